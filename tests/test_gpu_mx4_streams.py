"""GPU tests of the MX4 wrappers on another stream than the current one, while
work is pending there that still reads freed memory."""
import ctypes

import pytest
import torch

import mx4_reference as ref
from test_gpu_mx4 import _assert_mx4, _normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


T, O, K = 1000, 2100, 1000


def _operands(z):
    x, dy = _normal(T, K, "bf16", 1), _normal(T, O, "bf16", 2)
    w = z.mx4_quantize(_normal(O, K, "bf16", 3, 0.02))
    tight = z.MX4(w.codes, torch.cat([w.scales[:, :ref.blocks_of(K)], w.scales[:, :1]], 1).contiguous(), O, K)
    return dict(x=x, dy=dy, w=w, tight=tight, xq=z.mx4_quantize(x))


CALLS = {
    "quantize": lambda z, o, **kw: z.mx4_quantize(o["x"], **kw),
    "quantize columns": lambda z, o, **kw: z.mx4_quantize(o["x"], transpose=True, **kw),
    "quantize both": lambda z, o, **kw: z.mx4_quantize_both(o["x"], **kw),
    "transpose": lambda z, o, **kw: z.mx4_transpose(o["w"], **kw),
    "dequantize": lambda z, o, **kw: z.mx4_dequantize(o["w"], **kw),
    "matmul": lambda z, o, **kw: z.mx4_matmul(o["xq"], o["tight"], **kw),
    "linear": lambda z, o, **kw: z.mx4_linear(o["x"], o["tight"], **kw),
    "backward": lambda z, o, **kw: z.mx4_linear_backward(o["dy"], o["x"], o["w"], **kw),
}


def _tensors(results):
    """(An MX4 matrix's own bytes: what pads a row of scales is not written.)"""
    results = results if isinstance(results, tuple) else (results,)
    return [t for r in results
            for t in ((r,) if isinstance(r, torch.Tensor) else (r.codes, r.scales[:, :ref.blocks_of(r.cols)]))]


def _clone(results):
    return [t.clone() for t in _tensors(results)]


def _sizes(z, o):
    """Bytes of the blocks that the call takes."""
    n, sizes = ctypes.c_int64(), [4096]
    for w in (o["w"], o["tight"]):
        for query in (lambda: z.zero_mx4_linear_workspace(T, w._c, n), lambda: z.zero_mx4_matmul_workspace(o["xq"]._c, w._c, n),
                      lambda: z.zero_mx4_linear_backward_workspace(T, w._c, n)):
            assert query() == 0
            sizes.append(n.value)
    for rows, cols in ((T, K), (K, T), (O, K), (K, O)):
        nb = ref.blocks_of(cols)
        sizes.append(rows * (16 * nb + -(-nb // 16) * 16))
    return sizes + [2 * T * O, 2 * O * K, 2 * T * K]


@pytest.mark.parametrize("name", list(CALLS))
def test_pending_work_of_the_current_stream_keeps_its_memory(z, name):
    """Blocks of the sizes that the call takes are freed on the current stream
    while a copy of each still waits in its queue; the call on another stream
    must neither get those blocks at once nor be written over by what follows
    there."""
    o = _operands(z)
    want = _clone(CALLS[name](z, o))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in _sizes(z, o) if n]
    copies = [torch.empty_like(t) for t in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms: the call below runs meanwhile
    for c, t in zip(copies, freed):
        c.copy_(t)
    del freed, c, t
    for stream in (side, side.cuda_stream):
        got = CALLS[name](z, o, stream=stream)
        side.synchronize()
        for a, b in zip(_tensors(got), want):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    for c in copies:
        assert (c == 7).all()


def test_a_result_outlives_the_current_streams_reads(z):
    """A result made on another stream, read on the current one and freed while
    that read still waits: the next call on that stream must not write it."""
    x, other = _normal(T, K, "bf16", 1), _normal(T, K, "bf16", 2)
    side = torch.cuda.Stream()
    want = ref.quantize(x)
    z.mx4_quantize(other)
    torch.cuda.synchronize()
    m = z.mx4_quantize(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    codes, scales = m.codes.clone(), m.scales.clone()
    del m
    late = [z.mx4_quantize(other, stream=side) for _ in range(3)]
    torch.cuda.synchronize()
    _assert_mx4(z.MX4(codes, scales, T, K), *want, "read before it was freed")
    for m in late:
        _assert_mx4(m, *ref.quantize(other), "made after it")


@pytest.mark.parametrize("name", list(CALLS))
def test_operands_freed_after_the_call(z, name):
    """The operands are freed while the call still waits on its stream, and
    the current stream's next tensors are written at once."""
    o = _operands(z)
    want = _clone(CALLS[name](z, o))
    side = torch.cuda.Stream()
    sizes = [2 * T * K, 2 * T * O, O * K, T * K] + [t.untyped_storage().nbytes() for m in (o["w"], o["tight"], o["xq"])
                                                    for t in (m.codes, m.scales)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms: what follows here runs meanwhile
    got = CALLS[name](z, o, stream=side)
    del o
    late = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(_tensors(got), want):
        assert torch.equal(a, b)
    assert all((t == 7).all() for t in late)


@pytest.mark.parametrize("whole", [True, False])
def test_a_collectives_buffers_freed_after_the_call(z, whole):
    """The ranks' gradients, as one tensor or one a rank, freed while the
    reduce-scatter still waits on its stream."""
    n, ranks = 1 << 20, 4
    opt = z.ZeroOptimizer([n], [0], ranks, z.ZERO_STAGE_2, grad_buffers=False)
    opt.load_master()

    def gradients():
        m = z.mx4_quantize(_normal(ranks, n, "f32", 5, 0.01))
        codes, scales = m.codes.clone(), m.scales[:, :n // 32].contiguous()
        return (codes, scales) if whole else ([c.clone() for c in codes], [s.clone() for s in scales])

    shard = opt.view(z.ZERO_VIEW_GRAD_SHARD)
    opt.reduce_scatter_mx4(0, n, *gradients())
    want = shard[:n].clone()
    shard.zero_()
    side = torch.cuda.Stream()
    codes, scales = gradients()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    opt.reduce_scatter_mx4(0, n, codes, scales, stream=side)
    del codes, scales
    late = [torch.full((b,), 7, dtype=torch.uint8, device="cuda") for b in (ranks * n // 2, ranks * n // 32, n // 2, n // 32)
            for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(shard[:n], want) and all((t == 7).all() for t in late)
    opt.close()


def test_inside_a_captured_graph(z):
    """A forked stream of a capture: its memory comes from the graph's pool."""
    o = _operands(z)
    want = [_clone(CALLS[n](z, o)) for n in ("linear", "backward")]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        y = z.mx4_linear(o["x"], o["tight"], stream=side)
        grads = z.mx4_linear_backward(o["dy"], o["x"], o["w"])
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0][0])
        for a, b in zip(grads, want[1]):
            assert torch.equal(a, b)
