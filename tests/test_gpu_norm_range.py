"""GPU tests of the root-mean-square norm over the whole range of its types:
rows whose squares, or their sum, leave binary32's range at either end."""
import pytest
import torch

import layer_reference as ref
from test_gpu_mx8 import DTYPES, assert_mx8, normal
from test_gpu_rms_norm import _rstd_off, _weight

pytestmark = pytest.mark.gpu
U = ref.U


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def _far_rows(rows, cols, dtype):
    """Every other row far out: about 1e18, 1e19, 1e30 and the type's largest,
    and one large element among ordinary ones."""
    x = normal(rows, cols, dtype, cols).float()
    peak = x.abs().amax(1, keepdim=True)
    top = float(torch.finfo(DTYPES[dtype]).max)
    for k, size in enumerate((1.2e18, 1e19, 1e30, top)):
        x[2 * k + 1::10] = (x / peak)[2 * k + 1::10] * size
    x[9::10, cols // 2] = 1.9e19
    return x.to(DTYPES[dtype])


def _check_rows(n, h, w, eps=1e-6):
    """As for ordinary rows; a subnormal rstd is off by half of binary32's least
    step, and y, which is formed from it, by as much of itself."""
    y, rstd = ref.norm(h, w, eps)
    off = _rstd_off(h.shape[1])
    assert ((n.rstd.double() - rstd).abs() <= off * rstd + 2.0 ** -150).all()
    of_rstd = (2.0 ** -150 / rstd).unsqueeze(1)
    ref.assert_near(n.y, y, (off + of_rstd + 2.01 * U) * y.abs() + 2.0 ** -149, "y")


# a few lanes to a row, a warp with one vector a lane and with two, a block with
# one, two and four a thread, rows that are read twice; odd ones
SHAPES = [(40, 1), (40, 40), (43, 64), (40, 100), (40, 256), (3000, 512), (40, 512), (41, 771), (40, 2048), (700, 2048),
          (20, 5000), (20, 8192), (20, 12000), (20, 20000), (11, 20001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_whose_squares_are_past_binary32(z, shape, dtype):
    rows, cols = shape
    x, w = _far_rows(rows, cols, dtype), _weight(cols, dtype)
    n = z.rms_norm(x, w, h=True, y8=True, h8=True)
    _check_rows(n, x, w)
    assert n.y.abs().amax(1).min() > 0
    assert_mx8(n.y8, n.y, "y8")
    assert_mx8(n.h8, x, "h8")
    # the rows between them: the bits that they have without such neighbours
    near = x.clone()
    near[1::2] = 1
    want = z.rms_norm(near, w)
    assert torch.equal(n.y[0::2], want.y[0::2]) and torch.equal(n.rstd[0::2], want.rstd[0::2])
    # and in place
    over = x.clone()
    z.rms_norm(over, w, y=over)
    assert torch.equal(over, n.y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [64, 771, 2048, 20000])
def test_a_sum_with_the_residual_that_is_past_binary32(z, cols, dtype):
    x, r, w = _far_rows(12, cols, dtype), normal(12, cols, dtype, 3), _weight(cols, dtype)
    x[7::10] *= 0.25  # the largest stay finite
    r[3::10] *= 1e18
    n = z.rms_norm(x, w, residual=r)
    h = (x.float() + r.float()).to(x.dtype)
    assert torch.equal(n.h, h)
    _check_rows(n, h, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [1e-44, 1e-40, 2e-38])
@pytest.mark.parametrize("cols", [40, 256, 771, 2048, 12000, 20000])
def test_small_rows_and_a_small_eps(z, cols, eps, dtype):
    """eps below binary32's normal numbers: the squares below them count too."""
    x, w = normal(12, cols, dtype, 5).float(), _weight(cols, dtype)
    for k, size in enumerate((1e-14, 1e-18, 1e-20, 1e-22, 1e-30)):
        x[2 * k + 1] *= size
    x[11] = 0
    x = x.to(DTYPES[dtype])
    n = z.rms_norm(x, w, eps)
    _check_rows(n, x, w, float(torch.tensor(eps, dtype=torch.float32)))


def test_an_eps_near_binary32s_end(z):
    x, w = normal(4, 300, "f32", 1), _weight(300, "f32")
    x[1] = x[1] / x[1].abs().max() * 1.8e19
    for eps in (3.4e38, 1e30):
        n = z.rms_norm(x, w, eps)
        _check_rows(n, x, w, float(torch.tensor(eps, dtype=torch.float32)))


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [64, 100, 771, 2048, 5000])
def test_gradients_of_such_rows(z, cols, dtype, kept):
    """From the forward pass's own rstd.  (dx is of the order of rstd: of the
    furthest rows below binary32's normal numbers.)"""
    h, w, dy = _far_rows(40, cols, dtype), _weight(cols, dtype), normal(40, cols, dtype, 2, 0.1)
    n = z.rms_norm(h, w, h8=True)
    dx, dw = z.rms_norm_backward(dy, n.h8 if kept else h, w, n.rstd)
    value = z.mx8_dequantize(n.h8, torch.float32) if kept else h
    want_dx, want_dw, off_dx, off_dw = ref.norm_backward(dy, value, w, n.rstd)
    ref.assert_near(dx, want_dx, off_dx + 2.0 ** -149, "dx")
    ref.assert_near(dw, want_dw, off_dw, "dw")
    assert dw.abs().min() > 0


def test_infinities_and_nan_are_as_they_were(z):
    """An infinite element is no overflow of the squares: rstd is 0."""
    for cols in (64, 771, 4096, 17000):
        x, w = _far_rows(12, cols, "bf16"), _weight(cols, "bf16")
        clean = z.rms_norm(x, w)
        x[0, 3], x[1, 3], x[3, cols - 1], x[5, 0] = float("inf"), float("-inf"), float("nan"), float("inf")
        x[5, 1] = float("nan")
        n = z.rms_norm(x, w)
        assert (n.rstd[:2] == 0).all() and torch.isnan(n.rstd[[3, 5]]).all()
        assert torch.isnan(n.y[[0, 1], 3]).all() and not n.y[0, 4:].any()
        keep = [2, 4, 6, 7, 8, 9, 10, 11]
        assert torch.equal(n.y[keep], clean.y[keep]) and torch.equal(n.rstd[keep], clean.rstd[keep])
