"""GPU tests of the norm, its gradients and checkpoints as they are used --
captured, on two streams at once, right between writers of their operands -- at
the sizes that go other ways than a row of 256 columns: narrow, odd and long
rows, of which the gradients take three launches and a workspace, and rows far
out of binary32's range."""
import pytest
import torch

from test_gpu_layer_use import _clone, _same, _tensors
from test_gpu_mx8 import normal

pytestmark = pytest.mark.gpu
ROWS = 210


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def _operands(z, cols, seed=1):
    o = {k: normal(ROWS, cols, "bf16", seed + i, 0.3) for i, k in enumerate(("x", "r", "dy", "dh"))}
    o["x"][::7] *= 1e30
    o["w"] = 1 + normal(1, cols, "bf16", seed + 4, 0.1)[0]
    n = z.rms_norm(o["x"], o["w"], h8=True)
    return dict(o, x8=n.h8, rstd=n.rstd)


CALLS = {
    "norm": lambda z, o: z.rms_norm(o["x"], o["w"], residual=o["r"], y8=True, h8=True),
    "gradients": lambda z, o: z.rms_norm_backward(o["dy"], o["x"], o["w"], o["rstd"], dh=o["dh"]),
    "gradients from the checkpoint": lambda z, o: z.rms_norm_backward(o["dy"], o["x8"], o["w"], o["rstd"]),
    "quantise": lambda z, o: z.mx8_quantize(o["x"]),
    "read back": lambda z, o: z.mx8_dequantize(o["x8"]),
}
calls = pytest.mark.parametrize("name", list(CALLS))
sizes = pytest.mark.parametrize("cols", [40, 100, 771, 4096, 4101, 6144, 20000])


def _copy(o, new):
    for k, v in new.items():
        if isinstance(v, torch.Tensor):
            o[k].copy_(v)
        else:
            o[k].codes.copy_(v.codes)
            o[k].scales.copy_(v.scales)


@calls
@sizes
def test_captured_and_replayed(z, cols, name):
    o, other = _operands(z, cols), _operands(z, cols, 50)
    first = _operands(z, cols)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        CALLS[name](z, o)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = CALLS[name](z, o)
        graphs.append((g, out, torch.cuda.Stream()))
    for new in (first, other):
        want = _clone(CALLS[name](z, new))
        _copy(o, new)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, _, stream in graphs:
                with torch.cuda.stream(stream):
                    g.replay()
        torch.cuda.synchronize()
        for _, out, _ in graphs:
            assert _same(_tensors(out), want)


@calls
@sizes
def test_two_streams_at_once(z, cols, name):
    both = _operands(z, cols), _operands(z, cols, 50)
    want = [_clone(CALLS[name](z, o)) for o in both]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for k, o in enumerate(both):
            with torch.cuda.stream(streams[k]):
                got[k].append(CALLS[name](z, o))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(_same(_tensors(r), want[k]) for r in got[k])


@calls
@sizes
def test_right_after_its_operands_are_written(z, cols, name):
    o, new = _operands(z, cols), _operands(z, cols, 50)
    want = _clone(CALLS[name](z, new))
    for _ in range(4):
        CALLS[name](z, o)
        _copy(o, new)
        got = CALLS[name](z, o)
        for v in o.values():
            if isinstance(v, torch.Tensor):
                v.zero_()
            else:
                v.codes.zero_()
        torch.cuda.synchronize()
        assert _same(_tensors(got), want)
