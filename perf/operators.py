"""Measured cases of the microscaled 4-bit (MX4) operators.

MX4 stores a matrix in blocks of 32 consecutive elements of a row: one scale
2^(s - 127) (a byte s, 255 = the block is not a number) and 32 elements of
4 bits, each one of +-{0, .5, 1, 1.5, 2, 3, 4, 6}, two to a byte with the even
element in the low half.  A block's scale exponent is floor(log2(max|x|)) - 2.

  quantize   a 16- or 32-bit matrix into MX4, along its rows or down its
             columns, to nearest even or stochastically, and read back
  reduce     the reduce-scatter of N ranks' MX4 gradients: their fp32 sum in
             rank order, times 1/N, into the owners' 16-bit shards
  gather     the all-gather of the owners' 16-bit parameters of one matrix
             into N ranks' MX4 buffers, and every rank's product with it
  forward    y = Q(x) W^T of a linear layer, W in MX4
  backward   dx = Q(dy) Q(W^T)^T and dw = Q(dy^T) Q(x^T)^T of that layer; each
             operand in blocks along the axis its product sums over

Where ``own`` is false ``run`` computes them from elementary torch operations
in 32 bits; where it is true it calls the library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a batch of activations of hidden 2048, quantised for the forward product
        dict(name="quantize_rows", op="quantize", rows=8192, cols=2048, dtype="bf16", columns=False, seed=-1),
        # an activation matrix of odd sizes, quantised down its columns as a weight gradient's operand
        dict(name="quantize_columns_odd", op="quantize", rows=1237, cols=771, dtype="f16", columns=True, seed=-1),
        # a 32-bit gradient of the hidden-2048 qkv matrix, rounded stochastically before it is sent
        dict(name="quantize_stochastic", op="quantize", rows=2048, cols=6144, dtype="f32", columns=False, seed=7),
        # four ranks' gradients of one 768 x 768 projection
        dict(name="reduce_small", op="reduce", numel=768 * 768, ranks=4, dtype="bf16"),
        # eight ranks' gradients of one whole hidden-2048 layer (qkv, projection, two mlp matrices)
        dict(name="reduce_layer", op="reduce", numel=12 * 2048 * 2048, ranks=8, dtype="bf16"),
        # four ranks' copies of a 768-wide qkv matrix, one token each
        dict(name="gather_token", op="gather", out=2304, inner=768, tokens=1, ranks=4, dtype="bf16"),
        # eight ranks' copies of a hidden-2048 mlp matrix, a micro-batch each
        dict(name="gather_batch", op="gather", out=8192, inner=2048, tokens=512, ranks=8, dtype="bf16"),
        # one token through a hidden-4096 qkv matrix
        dict(name="forward_token", op="forward", out=12288, inner=4096, tokens=1, dtype="bf16"),
        # a ragged batch through a matrix of odd sizes, binary16
        dict(name="forward_odd", op="forward", out=1000, inner=771, tokens=333, dtype="f16"),
        # a training batch through a hidden-2048 mlp matrix
        dict(name="forward_batch", op="forward", out=8192, inner=2048, tokens=8192, dtype="bf16"),
        # the backward pass of a ragged batch through a 768-wide qkv matrix
        dict(name="backward_odd", op="backward", out=2304, inner=768, tokens=1003, dtype="bf16"),
        # the backward pass of a training batch through a hidden-4096 projection
        dict(name="backward_batch", op="backward", out=4096, inner=4096, tokens=8192, dtype="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "reduce", "gather", "forward", "backward"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "quantize":
        return dict(op=op, rows=_between(rng, 64, 8192), cols=_between(rng, 64, 8192), columns=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f16", "f32"]), seed=rng.choice([-1, rng.randrange(1 << 40)]))
    if op == "reduce":  # the flat space's intervals are multiples of 8 elements
        return dict(op=op, numel=8 * _between(rng, 1 << 14, 1 << 22), ranks=rng.choice([2, 3, 4, 8, 11, 16]), dtype=dtype)
    if op == "gather":  # a matrix of the flat space: whole blocks to a row
        return dict(op=op, out=8 * _between(rng, 32, 1024), inner=32 * _between(rng, 4, 128), dtype=dtype,
                    tokens=_between(rng, 1, 600), ranks=rng.choice([2, 3, 4, 8]))
    if op == "forward":
        return dict(op=op, out=_between(rng, 256, 16384), inner=_between(rng, 256, 8192), tokens=_between(rng, 1, 2048),
                    dtype=dtype)
    return dict(op=op, out=_between(rng, 256, 8192), inner=_between(rng, 256, 4096), tokens=_between(rng, 32, 2048),
                dtype=dtype)


def work(case):
    """Inputs read once, outputs written once (4.25 bits to an MX4 element)."""
    mx = (4 + 8 / BLOCK) / 8
    op = case["op"]
    if op == "quantize":
        # the matrix, its MX4 form written and read back, the values
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * BYTES[case["dtype"]] + 2 * mx), "flops": 0}
    if op == "reduce":
        return {"bytes": case["numel"] * (case["ranks"] * mx + 2), "flops": case["numel"] * (case["ranks"] + 1)}
    o, k, t = case["out"], case["inner"], case["tokens"]
    if op == "gather":
        n = case["ranks"]
        return {"bytes": o * k * (2 + n * mx) + 2 * n * t * (o + k), "flops": 2 * n * t * o * k}
    if op == "forward":
        return {"bytes": o * k * mx + 2 * t * (o + k), "flops": 2 * t * o * k}
    return {"bytes": o * k * (mx + 2) + 2 * t * (o + 2 * k), "flops": 4 * t * o * k}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols, dtype):
    """Normal, a few columns far larger, the last rows (padding) zero."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(3.0 * (torch.rand(cols, generator=g, device="cuda") < 0.02))
    x[rows - rows // 16:] = 0
    return x.to(DTYPES[dtype])


def _gradients(g, *shape):
    """Normal of deviation 1e-2 with one element in a hundred zero."""
    x = 1e-2 * torch.randn(*shape, generator=g, device="cuda")
    return x * (torch.rand(*shape, generator=g, device="cuda") >= 0.01)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case)
    if op == "quantize":
        x = _gradients(g, case["rows"], case["cols"]) if case["seed"] >= 0 else \
            _activations(g, case["rows"], case["cols"], "f32")
        st["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "reduce":
        n, ranks = case["numel"], case["ranks"]
        st["codes"], st["scales"] = _pack(*_quantize(_gradients(g, ranks, n)), n)
        if own:  # the optimizer that the program holds
            st["opt"] = _optimizer(case, n, "stage2")
            st["shard"] = _shard(st["opt"], case)
    elif op == "gather":
        o, k, ranks = case["out"], case["inner"], case["ranks"]
        st["w"] = (0.02 * torch.randn(o, k, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
        st["x"] = _activations(g, ranks * case["tokens"], k, case["dtype"]).view(ranks, case["tokens"], k)
        st["codes"] = torch.empty(ranks, o, k // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(ranks, o, k // BLOCK, dtype=torch.uint8, device="cuda")
        if own:
            st["opt"] = _optimizer(case, o * k, "stage3", st["w"])
    else:
        o, k, t = case["out"], case["inner"], case["tokens"]
        st["codes"], st["scales"] = _pack(*_quantize(0.02 * torch.randn(o, k, generator=g, device="cuda")), k)
        st["x"] = _activations(g, t, k, case["dtype"])
        if op == "backward":
            st["dy"] = _gradients(g, t, o).to(DTYPES[case["dtype"]])
    return st


# -------------------------------------------------------------- plain form --

def _random16(blocks, seed):
    """The 32 sixteen-bit numbers of each of `blocks` blocks: Philox4x32-10
    (Salmon, Moraes, Dror and Shaw 2011) keyed by the seed; call c of block b
    has the counter 4 b + c and gives the numbers of elements 8c .. 8c + 7,
    the low half of each word first."""
    m = 0xFFFFFFFF
    n = torch.arange(4 * blocks, dtype=torch.int64, device="cuda")
    c0, c1, c2, c3 = n & m, n >> 32, torch.zeros_like(n), torch.zeros_like(n)
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(10):  # the generator's rounds
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((q >> 32) & m) ^ c1 ^ k0, q & m, ((p >> 32) & m) ^ c3 ^ k1, p & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    w = torch.stack([c0, c1, c2, c3], -1)
    return torch.stack([w & 0xFFFF, w >> 16], -1).view(blocks, BLOCK)


def _power(e):
    """2^e in 32 bits, e a whole number from -127 to 127 (the least is subnormal)."""
    return torch.where(e == -127, 0x400000, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantize(x, seed=-1):
    """(signed element values, scale bytes) of the rows of x, in blocks along
    the last axis; the last block of a row is filled up with zeros."""
    cols = x.shape[-1]
    nb = -(-cols // BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - cols)).view(*x.shape[:-1], nb, BLOCK)
    e = x.abs().amax(-1).view(torch.int32) >> 23
    s = torch.where(e == 255, 255, (e - 2).clamp(min=0))
    a = torch.where(s == 255, 0.0, _power((127 - s).clamp(min=-127))).unsqueeze(-1) * x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    if seed >= 0:
        r = _random16(s.numel(), seed).view(a.shape)
        q = ((a / step * 65536).to(torch.int64) + r) >> 16
    else:
        q = torch.round(a / step)  # to nearest even
    v = torch.where((s == 255).unsqueeze(-1), 0.0, (q * step).clamp(max=6.0))
    return torch.copysign(v, x), s


def _pack(v, s, cols):
    """MX4 bytes of _quantize's result."""
    a = v.abs()
    c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = c | (torch.signbit(v).to(torch.uint8) << 3)
    c = c.flatten(-2)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), s.to(torch.uint8).contiguous()


def _values(v, s, cols):
    """The values that (elements, scale bytes) stand for."""
    scale = torch.where(s == 255, float("nan"), _power((s - 127).clamp(max=127)))
    return (v * scale.unsqueeze(-1)).flatten(-2)[..., :cols]


def _read(codes, scales, cols):
    """The values of MX4 bytes."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
    k = c & 7
    a = torch.where(k < 4, 0.5 * k, torch.where(k < 6, k - 2.0, 2.0 * k - 8.0))
    v = torch.where(c >= 8, -a, a)
    return _values(v.view(*scales.shape, BLOCK), scales.to(torch.int32), cols)


def _rounded(x, seed=-1):
    return _values(*_quantize(x, seed), x.shape[-1])


def _plain(st):
    op, dtype = st["op"], DTYPES[st["dtype"]]
    if op == "quantize":
        return _rounded(st["x"].t() if st["columns"] else st["x"], st["seed"]).to(dtype)
    if op == "reduce":
        g = _read(st["codes"], st["scales"], st["numel"])
        return (g.sum(0) * (1.0 / st["ranks"])).to(dtype)
    if op == "gather":
        w = _rounded(st["w"]).expand(st["ranks"], -1, -1).contiguous()
        return list(torch.matmul(_rounded(st["x"]), w.transpose(1, 2)).to(dtype).unbind(0))
    w = _read(st["codes"], st["scales"], st["inner"])
    if op == "forward":
        return torch.matmul(_rounded(st["x"]), w.t()).to(dtype)
    dx = torch.matmul(_rounded(st["dy"]), _rounded(w.t()).t())
    dw = torch.matmul(_rounded(st["dy"].t()), _rounded(st["x"].t()).t())
    return {"dx": dx.to(dtype), "dw": dw.to(dtype)}


# ------------------------------------------------------- the library's form --

def _optimizer(case, numel, stage, params=None):
    """The optimizer context of a program that holds `numel` parameters."""
    import zero_sharded_optimizer_sm_b200 as z

    opt = z.ZeroOptimizer([numel], [0], case["ranks"], z.ZERO_STAGE_2 if stage == "stage2" else z.ZERO_STAGE_3,
                          grad_buffers=False, dtype=z.ZERO_DTYPE_F16 if case["dtype"] == "f16" else z.ZERO_DTYPE_BF16)
    master = opt.view(z.ZERO_VIEW_MASTER)
    master.zero_()
    if params is not None:
        master[:numel] = params.reshape(-1)
    opt.load_master()
    return opt


def _shard(opt, case):
    import zero_sharded_optimizer_sm_b200 as z

    return opt.view(z.ZERO_VIEW_GRAD_SHARD)[:case["numel"]].view(DTYPES[case["dtype"]])


def _library(st):
    import zero_sharded_optimizer_sm_b200 as z

    op = st["op"]
    if op == "quantize":
        q = z.mx4_quantize(st["x"], transpose=st["columns"], seed=st["seed"] if st["seed"] >= 0 else None)
        return z.mx4_dequantize(q, st["x"].dtype)
    if op == "reduce":
        st["opt"].reduce_scatter_mx4(0, st["numel"], st["codes"], st["scales"])
        return st["shard"]
    if op == "gather":
        o, k = st["out"], st["inner"]
        st["opt"].all_gather_mx4(0, o * k, st["codes"], st["scales"])
        return [z.mx4_linear(x, z.MX4(c, s, o, k)) for x, c, s in zip(st["x"], st["codes"], st["scales"])]
    w = z.MX4(st["codes"], st["scales"], st["out"], st["inner"])
    if op == "forward":
        return z.mx4_linear(st["x"], w)
    dx, dw = z.mx4_linear_backward(st["dy"], st["x"], w)
    return {"dx": dx, "dw": dw}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------ in 64 bits ----

def _exact_numbers(blocks, seed):
    """The generator of _random16 on the host, in unsigned 64-bit numbers."""
    m = np.uint64(0xFFFFFFFF)
    h = np.uint64(32)
    n = np.arange(4 * blocks, dtype=np.uint64)
    ctr = [n & m, n >> h, np.zeros_like(n), np.zeros_like(n)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p = ctr[0] * np.uint64(0xD2511F53)
        q = ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(q >> h) ^ ctr[1] ^ np.uint64(key[0]), q & m, (p >> h) ^ ctr[3] ^ np.uint64(key[1]), p & m]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    half = np.stack([part for w in ctr for part in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1)
    return torch.from_numpy(half.reshape(blocks, BLOCK).astype(np.float64)).cuda()


GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 8.0)


def _exact_power(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round(x, seed=-1):
    """The MX4 values of x's rows: the grid's two neighbours of each element,
    and the choice between them."""
    x = x.double()
    cols = x.shape[-1]
    nb = -(-cols // BLOCK)
    padded = torch.zeros(*x.shape[:-1], nb * BLOCK, dtype=torch.float64, device=x.device)
    padded[..., :cols] = x
    blocks = padded.view(*x.shape[:-1], nb, BLOCK)
    top = blocks.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
    unit = _exact_power(torch.where(top > 0, e - 3, -127).clamp(min=-127))
    a = blocks.abs() / unit
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    at = torch.bucketize(a, grid, right=True) - 1  # grid[at] <= a < grid[at + 1]
    low, high = grid[at], grid[at + 1]
    if seed >= 0:
        part = torch.floor((a - low) / (high - low) * 65536)
        up = part + _exact_numbers(a.numel() // BLOCK, seed).view(a.shape) >= 65536
    else:
        twice = 2 * a - (low + high)
        up = (twice > 0) | ((twice == 0) & (at % 2 == 1))
    v = torch.where(up, high, low).clamp(max=6.0) * unit
    return (v * torch.sign(blocks)).flatten(-2)[..., :cols]


def _exact_read(codes, scales, cols):
    table = torch.tensor(GRID[:8] + tuple(-v for v in GRID[:8]), dtype=torch.float64, device="cuda")
    v = torch.empty(*codes.shape, 2, dtype=torch.float64, device="cuda")
    v[..., 0] = table[(codes % 16).long()]
    v[..., 1] = table[(codes // 16).long()]
    unit = _exact_power(scales.to(torch.int64) - 127).unsqueeze(-1)
    return (v.view(*scales.shape, BLOCK) * unit).flatten(-2)[..., :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_round(st["x"].t() if case["columns"] else st["x"], case["seed"])
    if op == "reduce":
        return sum(_exact_read(c, s, case["numel"]) for c, s in zip(st["codes"], st["scales"])) / case["ranks"]
    if op == "gather":
        w = _exact_round(st["w"])
        return [_exact_round(x) @ w.t() for x in st["x"]]
    w = _exact_read(st["codes"], st["scales"], case["inner"])
    if op == "forward":
        return _exact_round(st["x"]) @ w.t()
    return {"dx": _exact_round(st["dy"]) @ _exact_round(w.t()).t(),
            "dw": _exact_round(st["dy"].t()) @ _exact_round(st["x"].t()).t()}
