"""Measured cases of the operators around a layer's 4-bit products in a
training step: what the backward pass keeps, the norm, the embedding.

An MX8 matrix keeps its rows in blocks of 32 elements: one scale 2^(s - 127)
(a byte s, 255 = the block is not a number) and 32 elements of 8 bits (four
exponent and three mantissa bits, at most 448).  s is the smallest with
max|x| <= 448 * 2^(s - 127), from 3 to 246.  MX4 is the 4-bit format of
perf/operators.py.

  checkpoint          an activation into MX8, and read back
  saved               the backward pass of a linear layer with an MX4 weight
                      whose input was kept in MX8
  norm                h = x + residual, y = h * (mean(h^2) + eps)^-1/2 * weight,
                      and both in MX8
  norm_backward       its gradients, from h or from h in MX8
  embedding           rows of a table (16-bit, or a gathered MX4 one) by token,
                      scaled; tokens below 0 are padding and give zeros
  embedding_backward  the table's whole gradient

Where ``own`` is false ``run`` computes them from elementary torch operations
in 32 bits (sums over many rows or a row's squares in 64); where it is true it
calls the library.
"""
import math

import torch

own = False

BLOCK = 32
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
MX4_BYTES, MX8_BYTES = 17 / 32, 33 / 32  # of an element


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a short prompt's activations of hidden 768, kept for the backward pass
        dict(name="checkpoint_small", op="checkpoint", rows=128, cols=768, dtype="bf16"),
        # a training batch's activations of hidden 4096
        dict(name="checkpoint_batch", op="checkpoint", rows=8192, cols=4096, dtype="bf16"),
        # a ragged batch back through a 768-wide qkv matrix
        dict(name="saved_odd", op="saved", out=2304, inner=768, tokens=1003, dtype="bf16"),
        # a training batch back through the hidden-2048 qkv matrix
        dict(name="saved_batch", op="saved", out=6144, inner=2048, tokens=8192, dtype="bf16"),
        # one token of hidden 4096, as when serving: nothing is kept
        dict(name="norm_token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, mx8=False),
        # a training batch of hidden 4096, with everything that the backward pass reads
        dict(name="norm_batch", op="norm", rows=8192, cols=4096, dtype="bf16", residual=True, mx8=True),
        # odd sizes in binary16, the norm's input kept as it was
        dict(name="norm_backward_odd", op="norm_backward", rows=1237, cols=771, dtype="f16", residual=False, mx8=False),
        # the backward pass of norm_batch, from the 8-bit checkpoint, with the residual stream's own gradient
        dict(name="norm_backward_batch", op="norm_backward", rows=8192, cols=4096, dtype="bf16", residual=True, mx8=True),
        # a ragged batch from a binary16 table of odd sizes
        dict(name="embedding_odd", op="embedding", tokens=1003, vocab=32001, cols=771, dtype="f16", mx4=False),
        # a training batch from a hidden-4096 table that was gathered in MX4
        dict(name="embedding_gathered", op="embedding", tokens=8192, vocab=32000, cols=4096, dtype="bf16", mx4=True),
        # one short sequence into a small hidden-768 table
        dict(name="embedding_backward_small", op="embedding_backward", tokens=301, vocab=5003, cols=768, dtype="f16"),
        # a training batch into a hidden-2048 table
        dict(name="embedding_backward_batch", op="embedding_backward", tokens=16384, vocab=50304, cols=2048, dtype="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["checkpoint", "saved", "norm", "norm_backward", "embedding", "embedding_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "saved":
        return dict(op=op, out=_between(rng, 256, 6144), inner=_between(rng, 256, 2048), tokens=_between(rng, 32, 2048),
                    dtype=rng.choice(["bf16", "bf16", "f16"]))
    if op in ("embedding", "embedding_backward"):
        cols = _between(rng, 64, 4096)
        case = dict(op=op, tokens=_between(rng, 1, 8192), vocab=_between(rng, 256, (1 << 26) // cols), cols=cols,
                    dtype=dtype)
        return dict(case, mx4=rng.random() < 0.5) if op == "embedding" else case
    cols = _between(rng, 32, 8192)
    case = dict(op=op, rows=_between(rng, 1, min(1 << 15, (1 << 24) // cols)), cols=cols, dtype=dtype)
    return case if op == "checkpoint" else dict(case, residual=rng.random() < 0.5, mx8=rng.random() < 0.5)


def work(case):
    """Inputs read once, outputs written once; what is kept in MX8 is read back
    to be looked at."""
    op, b = case["op"], BYTES[case["dtype"]]
    if op == "saved":
        o, k, t = case["out"], case["inner"], case["tokens"]
        return {"bytes": o * k * (MX4_BYTES + b) + t * (b * (o + k) + MX8_BYTES * k), "flops": 4 * t * o * k}
    if op == "embedding":
        t, cols = case["tokens"], case["cols"]
        rows = min(_distinct(t, case["vocab"]), case["vocab"])
        return {"bytes": t * (8 + cols * b) + rows * cols * (MX4_BYTES if case["mx4"] else b), "flops": t * cols}
    if op == "embedding_backward":
        t, cols = case["tokens"], case["cols"]
        return {"bytes": t * (8 + cols * b) + case["vocab"] * cols * b, "flops": 2 * t * cols}
    n = case["rows"] * case["cols"]
    if op == "checkpoint":
        return {"bytes": n * 2 * (b + MX8_BYTES), "flops": 0}
    if op == "norm":
        each = 2 * b + 2 * b * case["residual"]  # x and y; the residual and h
        if case["mx8"]:
            each += 2 * (2 * MX8_BYTES + 2)      # y and h in MX8, read back in 16 bits
        return {"bytes": n * each + case["cols"] * b + 4 * case["rows"], "flops": 5 * n}
    each = 2 * b + b * case["residual"] + (MX8_BYTES if case["mx8"] else b)
    return {"bytes": n * each + 2 * case["cols"] * b + 4 * case["rows"], "flops": 9 * n}


def _distinct(tokens, vocab):
    """About how many different tokens _tokens gives: of weight 1 / v each."""
    total, v, sum_ = math.log(vocab + 1), 1, 0.0
    while v <= vocab:  # by octaves
        n = min(v, vocab - v + 1)
        sum_ += n * -math.expm1(-tokens / (total * 1.5 * v))
        v *= 2
    return max(1, int(sum_))


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


def _gradients(g, rows, cols, dtype):
    """Normal of deviation 1e-2 with one element in a hundred zero."""
    x = 1e-2 * torch.randn(rows, cols, generator=g, device="cuda")
    return (x * (torch.rand(rows, cols, generator=g, device="cuda") >= 0.01)).to(DTYPES[dtype])


def _tokens(g, n, vocab):
    """Token v with weight 1 / (v + 1); a sixteenth at the end is padding."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(vocab + 1)) - 1).to(torch.int64).clamp(max=vocab - 1)
    t[n - n // 16:] = -1
    return t


def prepare(case, seed):
    g = _generator(seed)
    op, dtype = case["op"], case["dtype"]
    st = dict(case)
    if op == "checkpoint":
        st["x"] = _activations(g, case["rows"], case["cols"], dtype)
    elif op == "saved":
        o, k, t = case["out"], case["inner"], case["tokens"]
        st["codes"], st["scales"] = _pack4(*_quantize4(0.02 * torch.randn(o, k, generator=g, device="cuda")))
        st["x_codes"], st["x_scales"] = _pack8(*_quantize8(_activations(g, t, k, dtype).float()))
        st["dy"] = _gradients(g, t, o, dtype)
    elif op == "embedding":
        v, cols = case["vocab"], case["cols"]
        table = 0.02 * torch.randn(v, cols, generator=g, device="cuda")
        if case["mx4"]:
            st["codes"], st["scales"] = _pack4(*_quantize4(table))
        else:
            st["table"] = table.to(DTYPES[dtype])
        st["t"] = _tokens(g, case["tokens"], v)
        st["scale"] = math.sqrt(cols)
    elif op == "embedding_backward":
        st["dy"] = _gradients(g, case["tokens"], case["cols"], dtype)
        st["t"] = _tokens(g, case["tokens"], case["vocab"])
        st["scale"] = math.sqrt(case["cols"])
    else:
        rows, cols = case["rows"], case["cols"]
        st["w"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[dtype])
        if op == "norm":
            st["x"] = _activations(g, rows, cols, dtype)
            st["r"] = _activations(g, rows, cols, dtype) if case["residual"] else None
        else:
            h = _activations(g, rows, cols, dtype)
            st["rstd"] = torch.rsqrt(h.double().square().mean(1) + EPS).float()
            if case["mx8"]:
                st["h_codes"], st["h_scales"] = _pack8(*_quantize8(h.float()))
            else:
                st["h"] = h
            st["dy"] = _gradients(g, rows, cols, dtype)
            st["dh"] = _gradients(g, rows, cols, dtype) if case["residual"] else None
    return st


# -------------------------------------------------------------- plain form --

def _power(e):
    """2^e in 32 bits, e a whole number from -127 to 127 (the least is subnormal)."""
    return torch.where(e == -127, 0x400000, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(x):
    """The rows of x in blocks, the last of a row filled up with zeros."""
    nb = -(-x.shape[1] // BLOCK)
    return torch.nn.functional.pad(x, (0, nb * BLOCK - x.shape[1])).view(x.shape[0], nb, BLOCK)


def _quantize4(x):
    """(signed element values, scale bytes) of the rows of a 32-bit x in MX4."""
    x = _blocks(x)
    e = x.abs().amax(-1).view(torch.int32) >> 23
    s = torch.where(e == 255, 255, (e - 2).clamp(min=0))
    a = torch.where(s == 255, 0.0, _power((127 - s).clamp(min=-127))).unsqueeze(-1) * x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), x), s


def _quantize8(x):
    """(signed element values, scale bytes) of the rows of a 32-bit x in MX8."""
    x = _blocks(x)
    top = x.abs().amax(-1).view(torch.int32)
    s = (((top + 0x1FFFFF) >> 23) - 8).clamp(3, 246)  # one more where the mantissa is over 448's
    s = torch.where(top >> 23 == 255, 255, s)
    a = torch.where(s == 255, 0.0, _power((127 - s).clamp(min=-127))).unsqueeze(-1) * x.abs()
    step = _power(((a.view(torch.int32) >> 23) - 127).clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x), s


def _pack4(v, s):
    """MX4 bytes of _quantize4's result."""
    a = v.abs()
    c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = (c | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), s.to(torch.uint8).contiguous()


def _pack8(v, s):
    """MX8 bytes of _quantize8's result."""
    return v.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2).contiguous(), s.to(torch.uint8).contiguous()


def _values(v, s, cols):
    """The values that (elements, scale bytes) stand for."""
    s = s.to(torch.int32)
    scale = torch.where(s == 255, float("nan"), _power((s - 127).clamp(max=127)))
    return (v * scale.unsqueeze(-1)).flatten(-2)[..., :cols]


def _read4(codes, scales, cols):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int32)
    k = c & 7
    a = torch.where(k < 4, 0.5 * k, torch.where(k < 6, k - 2.0, 2.0 * k - 8.0))
    return _values(torch.where(c >= 8, -a, a).view(*scales.shape, BLOCK), scales, cols)


def _read8(codes, scales, cols):
    return _values(codes.view(torch.float8_e4m3fn).float().view(*scales.shape, BLOCK), scales, cols)


def _rounded4(x):
    return _values(*_quantize4(x), x.shape[1])


def _rounded8(x):
    return _values(*_quantize8(x), x.shape[1])


def _plain(st):
    op, dtype = st["op"], DTYPES[st["dtype"]]
    if op == "checkpoint":
        return _rounded8(st["x"].float()).to(dtype)
    if op == "saved":
        w = _read4(st["codes"], st["scales"], st["inner"])
        x = _read8(st["x_codes"], st["x_scales"], st["inner"])
        dy = st["dy"].float()
        dx = torch.matmul(_rounded4(dy), _rounded4(w.t()).t())
        dw = torch.matmul(_rounded4(dy.t()), _rounded4(x.t()).t())
        return {"dx": dx.to(dtype), "dw": dw.to(dtype)}
    if op == "norm":
        h = st["x"]
        if st["r"] is not None:
            h = (h.float() + st["r"].float()).to(dtype)
        f = h.float()
        rstd = torch.rsqrt(f.double().square().mean(1) + EPS).float()
        y = (f * rstd.unsqueeze(1) * st["w"].float()).to(dtype)
        out = {"y": y}
        if st["r"] is not None:
            out["h"] = h
        if st["mx8"]:
            # (an MX8 value is exact in bfloat16)
            out.update(rstd=rstd, y8=_rounded8(y.float()).bfloat16(), h8=_rounded8(f).bfloat16())
        return out
    if op == "norm_backward":
        h = _read8(st["h_codes"], st["h_scales"], st["cols"]) if st["mx8"] else st["h"].float()
        rstd, dy = st["rstd"].unsqueeze(1), st["dy"].float()
        xh, g = h * rstd, dy * st["w"].float()
        c = (g * xh).double().mean(1, keepdim=True).float()
        dx = rstd * (g - xh * c)
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return {"dx": dx.to(dtype), "dw": (dy * xh).sum(0, dtype=torch.float64).to(dtype)}
    t = st["t"]
    there = t >= 0
    if op == "embedding":
        at = t.clamp(min=0)
        if st["mx4"]:
            rows = _read4(st["codes"][at], st["scales"][at], st["cols"])
        else:
            rows = st["table"][at].float()
        return (torch.where(there.unsqueeze(1), rows, 0.0) * st["scale"]).to(dtype)
    # padding goes to a row behind the table
    sums = torch.zeros(st["vocab"] + 1, st["cols"], device="cuda")
    sums.index_add_(0, torch.where(there, t, st["vocab"]), st["dy"].float())
    return (sums[:-1] * st["scale"]).to(dtype)


# ------------------------------------------------------- the library's form --

def _library(st):
    import zero_sharded_optimizer_sm_b200 as z

    op, dtype = st["op"], DTYPES[st["dtype"]]
    if op == "checkpoint":
        return z.mx8_dequantize(z.mx8_quantize(st["x"]), dtype)
    if op == "saved":
        w = z.MX4(st["codes"], st["scales"], st["out"], st["inner"])
        x = z.MX8(st["x_codes"], st["x_scales"], st["tokens"], st["inner"])
        dx, dw = z.mx4_linear_backward(st["dy"], x, w)
        return {"dx": dx, "dw": dw}
    if op == "norm":
        if not st["mx8"]:
            n = z.rms_norm(st["x"], st["w"], EPS, residual=st["r"], rstd=False)
            return {"y": n.y, "h": n.h} if st["r"] is not None else {"y": n.y}
        n = z.rms_norm(st["x"], st["w"], EPS, residual=st["r"], y8=True, h8=True)
        out = {"y": n.y, "rstd": n.rstd, "y8": z.mx8_dequantize(n.y8), "h8": z.mx8_dequantize(n.h8)}
        return dict(out, h=n.h) if st["r"] is not None else out
    if op == "norm_backward":
        h = z.MX8(st["h_codes"], st["h_scales"], st["rows"], st["cols"]) if st["mx8"] else st["h"]
        dx, dw = z.rms_norm_backward(st["dy"], h, st["w"], st["rstd"], dh=st["dh"])
        return {"dx": dx, "dw": dw}
    if op == "embedding":
        table = z.MX4(st["codes"], st["scales"], st["vocab"], st["cols"]) if st["mx4"] else st["table"]
        return z.embedding(st["t"], table, st["scale"], dtype=dtype)
    return z.embedding_backward(st["dy"], st["t"], st["vocab"], st["scale"])


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------ in 64 bits ----

GRID4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 8.0)


def _exact_power(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_blocks(x):
    nb = (x.shape[1] + BLOCK - 1) // BLOCK
    padded = torch.zeros(x.shape[0], nb * BLOCK, dtype=torch.float64, device=x.device)
    padded[:, :x.shape[1]] = x
    return padded.view(x.shape[0], nb, BLOCK)


def _exact_round(x, grid, exponent):
    """x's rows on `grid` in blocks of the scale 2^exponent(block maximum): the
    grid's two neighbours of each element, and the choice between them."""
    blocks = _exact_blocks(x)
    unit = _exact_power(exponent(blocks.abs().amax(-1, keepdim=True)))
    a = blocks.abs() / unit
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    at = torch.bucketize(a, grid, right=True) - 1  # grid[at] <= a < grid[at + 1]
    low, high = grid[at], grid[at + 1]
    twice = 2 * a - (low + high)
    up = (twice > 0) | ((twice == 0) & (at % 2 == 1))
    v = torch.where(up, high, low).clamp(max=float(grid[-2])) * unit
    return (v * torch.sign(blocks)).flatten(-2)[:, :x.shape[1]]


def _exact_round4(x):
    return _exact_round(x, GRID4, lambda top: torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127))


def _grid8():
    """The magnitudes of E4M3 in order, and one more above them."""
    sub = [i / 512 for i in range(8)]
    normal = [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]  # the last pattern is NaN
    return tuple(sub + normal + [480.0])


def _exact_round8(x):
    def exponent(top):  # the smallest e from -124 to 119 with top <= 448 * 2^e
        e = torch.frexp(top / 448)[1]
        return torch.where(top <= 448 * _exact_power(e - 1), e - 1, e).clamp(-124, 119)

    return _exact_round(x, _grid8(), exponent)


def _exact_read(elements, scales, cols):
    unit = _exact_power(scales.to(torch.int64) - 127).unsqueeze(-1)
    return (elements.view(*scales.shape, BLOCK) * unit).flatten(-2)[:, :cols]


def _exact_read4(codes, scales, cols):
    table = torch.tensor(GRID4[:8] + tuple(-v for v in GRID4[:8]), dtype=torch.float64, device="cuda")
    v = torch.empty(*codes.shape, 2, dtype=torch.float64, device="cuda")
    v[..., 0] = table[(codes % 16).long()]
    v[..., 1] = table[(codes // 16).long()]
    return _exact_read(v, scales, cols)


def _exact_read8(codes, scales, cols):
    half = _grid8()[:-1] + (float("nan"),)
    table = torch.tensor(half + tuple(-v for v in half), dtype=torch.float64, device="cuda")
    return _exact_read(table[codes.long()], scales, cols)


def exact(case, seed):
    st = prepare(case, seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op == "checkpoint":
        return _exact_round8(st["x"].double())
    if op == "saved":
        w = _exact_read4(st["codes"], st["scales"], case["inner"])
        x = _exact_read8(st["x_codes"], st["x_scales"], case["inner"])
        dy = st["dy"].double()
        return {"dx": _exact_round4(dy) @ _exact_round4(w.t()).t(),
                "dw": _exact_round4(dy.t()) @ _exact_round4(x.t()).t()}
    if op == "norm":
        x = st["x"].double()
        total = x if st["r"] is None else x + st["r"].double()
        h = total.to(dtype).double()  # the norm is of h as it is kept
        rstd = 1 / torch.sqrt(torch.einsum("rc,rc->r", h, h) / case["cols"] + EPS)
        y = torch.einsum("rc,r,c->rc", h, rstd, st["w"].double())
        out = {"y": y}
        if case["residual"]:
            out["h"] = total
        if case["mx8"]:
            out.update(rstd=rstd, y8=_exact_round8(y.to(dtype).double()), h8=_exact_round8(h))
        return out
    if op == "norm_backward":
        h = _exact_read8(st["h_codes"], st["h_scales"], case["cols"]) if case["mx8"] else st["h"].double()
        dy, w, rstd = st["dy"].double(), st["w"].double(), st["rstd"].double()
        dot = torch.einsum("rc,rc,c->r", dy, h, w)
        dx = torch.einsum("r,rc,c->rc", rstd, dy, w) - h * (rstd ** 3 * dot / case["cols"]).unsqueeze(1)
        if case["residual"]:
            dx = dx + st["dh"].double()
        return {"dx": dx, "dw": torch.einsum("rc,rc,r->c", dy, h, rstd)}
    t = st["t"]
    if op == "embedding":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        at = torch.nonzero(t >= 0).squeeze(1)
        if case["mx4"]:
            rows = _exact_read4(st["codes"][t[at]], st["scales"][t[at]], case["cols"])
        else:
            rows = st["table"][t[at]].double()
        out[at] = rows * st["scale"]
        return out
    # sums of runs of equal tokens, as differences of running sums
    order = torch.argsort(t, stable=True)
    running = torch.cat([torch.zeros(1, case["cols"], dtype=torch.float64, device="cuda"),
                         torch.cumsum(st["dy"].double()[order], 0)])
    ends = torch.searchsorted(t[order], torch.arange(-1, case["vocab"], device="cuda"), right=True)
    return (running[ends[1:]] - running[ends[:-1]]) * st["scale"]
