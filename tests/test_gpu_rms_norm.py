"""GPU tests of the root-mean-square norm and its gradients against the formulas
in 64 bits."""
import pytest
import torch

import layer_reference as ref
from test_gpu_mx8 import DTYPES, assert_mx8, normal

pytestmark = pytest.mark.gpu
U = ref.U


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def _weight(cols, dtype, seed=7):
    return (1 + 0.1 * normal(1, cols, "f32", seed)[0]).to(DTYPES[dtype])


# A row's sum of squares: a thread adds at most 32 of them one after another (in
# rows of more than 16384 columns cols / 512, rounded up to eights), and at most
# 10 more additions join the threads; a sum of positive terms is off by the
# additions on a term's way, the root by half of that, and the division by the
# columns, eps's addition, the root and the reciprocal round once each.
def _rstd_off(cols):
    chain = 32 if cols <= 16384 else 8 * -(-cols // 4096)
    return ((chain + 11) / 2 + 4) * U


def _check(z, x, r, w, eps=1e-6, **kw):
    n = z.rms_norm(x, w, eps, residual=r, h=True, y8=True, h8=True, **kw)
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(n.h, h)
    y, rstd = ref.norm(h, w, eps)
    off = _rstd_off(x.shape[1])
    assert ((n.rstd.double() - rstd).abs() <= off * rstd).all()
    ref.assert_near(n.y, y, (off + 2.01 * U) * y.abs() + 2.0 ** -149, "y")
    assert_mx8(n.y8, n.y, "y8")
    assert_mx8(n.h8, h, "h8")
    return n


SHAPES = [(1, 1), (1, 4096), (3, 7), (2, 33), (5, 256), (4, 257), (130, 771), (67, 768), (6, 1000), (9, 1024), (3, 1025),
          (33, 2048), (17, 2056), (65, 4096), (3, 5000), (2, 8192), (3, 8200), (2, 16384), (2, 16385), (3, 30011), (1, 200001),
          (1237, 100)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(z, shape, dtype, residual):
    rows, cols = shape
    x = normal(rows, cols, dtype, cols)
    x[rows // 2:] *= 30
    if rows > 2:
        x[-1] = 0
    r = normal(rows, cols, dtype, rows + cols) if residual else None
    if residual and rows > 2:
        r[-1] = 0  # a row of zeros: rstd is eps^-1/2, y is 0
    n = _check(z, x, r, _weight(cols, dtype))
    if rows > 2:
        assert not n.y[-1].any()


@pytest.mark.parametrize("wtype", list(DTYPES))
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("eps", [1e-12, 1e-5, 1.0])
def test_norm_types_of_weights_and_eps(z, dtype, wtype, eps):
    _check(z, normal(19, 300, dtype, 1), normal(19, 300, dtype, 2), _weight(300, wtype), eps)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [96, 300, 771, 2048, 4100, 20000])
def test_norm_of_strided_rows_in_place_and_one_result_alone(z, dtype, cols):
    rows, t = 7, DTYPES[dtype]
    for off, pad in ((0, 8), (1, 3), (8, 5)):
        space = normal(rows + 1, cols + pad, dtype, 3).flatten()
        x = space[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        r, w = normal(rows, cols, dtype, 4), _weight(cols, dtype)
        want = _check(z, x, r, w)
        # one result at a time
        assert torch.equal(z.rms_norm(x, w, residual=r, h=False, rstd=False).y, want.y)
        only = z.rms_norm(x, w, residual=r, y=False, rstd=False)
        assert torch.equal(only.h, want.h) and only.y is None and only.rstd is None and only.y8 is None
        only = z.rms_norm(x, w, residual=r, y=False, h=None, rstd=True)
        assert torch.equal(only.rstd, want.rstd)
        only = z.rms_norm(x, w, residual=r, y=False, h=False, rstd=False, y8=True)
        assert_mx8(only.y8, want.y, "y8 alone")
        only = z.rms_norm(x, w, residual=r, y=False, h=False, rstd=False, h8=True)
        assert_mx8(only.h8, want.h, "h8 alone")
        # in place: h over the residual, y over x; what lies between the rows stays
        before, both = space.clone(), r.clone()
        n = z.rms_norm(x, w, residual=both, y=x, h=both)
        assert n.y is x and n.h is both
        assert torch.equal(x, want.y) and torch.equal(both, want.h)
        rest = torch.ones_like(space, dtype=torch.bool)
        rest[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False
        assert torch.equal(space[rest], before[rest])
        # h over x, y over the residual
        a, b = normal(rows, cols, dtype, 5), normal(rows, cols, dtype, 6)
        want = z.rms_norm(a, w, residual=b)
        z.rms_norm(a, w, residual=b, y=b, h=a)
        assert torch.equal(b, want.y) and torch.equal(a, want.h)
    assert n.y.dtype == t


@pytest.mark.parametrize("cols", [64, 771, 4096, 17000])
def test_norm_of_rows_with_infinities_and_nan(z, cols):
    """They stay within their rows."""
    x = normal(6, cols, "bf16", 1)
    clean = z.rms_norm(x, _weight(cols, "bf16"), y8=True)
    y = x.clone()
    y[1, 5], y[4, cols - 1], y[4, 0] = float("nan"), float("inf"), float("-inf")
    n = z.rms_norm(y, _weight(cols, "bf16"), y8=True, h8=True)
    for row in (0, 2, 3, 5):
        assert torch.equal(n.y[row], clean.y[row]) and torch.equal(n.y8.codes[row], clean.y8.codes[row])
    assert torch.isnan(n.y[1]).all() and torch.isnan(n.rstd[1])
    assert n.rstd[4] == 0 and torch.isnan(n.y[4, [0, cols - 1]]).all() and not n.y[4, 1:cols - 1].any()
    assert_mx8(n.y8, n.y, "y8")
    assert_mx8(n.h8, y, "h8")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_norm_of_large_and_small_rows(z, dtype):
    """Values at the ends of binary16's range, and (f32) whose squares leave
    binary32's normal numbers below: rstd is then eps's."""
    x = normal(4, 512, dtype, 1).float()
    x[0] = x[0] / x[0].abs().max() * 60000
    x[1] *= 1e-25
    x[2] *= 1e-3
    _check(z, x.to(DTYPES[dtype]), None, _weight(512, "f32"))


def _check_backward(z, dy, h, w, dh, seed=0, **kw):
    _, rstd = ref.norm(h.double() if not isinstance(h, z.MX8) else z.mx8_dequantize(h, torch.float32).double(), w, 1e-6)
    rstd = rstd.float()
    dx, dw = z.rms_norm_backward(dy, h, w, rstd, dh=dh, **kw)
    value = z.mx8_dequantize(h, torch.float32) if isinstance(h, z.MX8) else h
    want_dx, want_dw, off_dx, off_dw = ref.norm_backward(dy, value, w, rstd, dh)
    ref.assert_near(dx, want_dx, off_dx, "dx")
    ref.assert_near(dw, want_dw, off_dw, "dw")
    return dx, dw


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES + [(2000, 768), (5000, 40)])
def test_norm_backward(z, shape, dtype, kept):
    rows, cols = shape
    h, dy = normal(rows, cols, dtype, 1), normal(rows, cols, dtype, 2, 0.1)
    if rows > 2:
        dy[-1] = 0
    dh = normal(rows, cols, dtype, 3, 0.1) if rows % 2 else None
    _check_backward(z, dy, z.mx8_quantize(h) if kept else h, _weight(cols, dtype), dh)


@pytest.mark.parametrize("wtype,dwtype", [("bf16", "f32"), ("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_norm_backward_types(z, dtype, wtype, dwtype):
    h, dy = normal(300, 520, dtype, 1), normal(300, 520, dtype, 2, 0.1)
    flat = torch.full((536,), 5.0, dtype=DTYPES[dwtype], device="cuda")  # a rank's gradient buffer
    got = _check_backward(z, dy, h, _weight(520, wtype), dy, dw=flat[8:528])
    assert got[0].dtype == dy.dtype and (flat[:8] == 5).all() and (flat[528:] == 5).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [96, 301, 771, 2048, 4100, 20000])
def test_norm_backward_of_strided_rows_and_in_place(z, dtype, cols):
    rows = 23
    for off, pad in ((0, 8), (1, 3)):
        space = normal(rows + 1, cols + pad, dtype, 3, 0.1).flatten()
        dy = space[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        h, dh, w = normal(rows, cols, dtype, 4), normal(rows, cols, dtype, 5, 0.1), _weight(cols, dtype)
        rstd = ref.norm(h, w, 1e-6)[1].float()
        want_dx, want_dw = _check_backward(z, dy, h, w, dh)
        over = dh.clone()
        dx, dw = z.rms_norm_backward(dy, h, w, rstd, dh=over, dx=over)
        assert dx is over and torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
        before = space.clone()
        dx, dw = z.rms_norm_backward(dy, h, w, rstd, dh=dh, dx=dy)
        assert torch.equal(dy, want_dx) and torch.equal(dw, want_dw)
        rest = torch.ones_like(space, dtype=torch.bool)
        rest[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False
        assert torch.equal(space[rest], before[rest])


def _laid(x, off, pitch):
    """The matrix `off` elements into memory of its own, rows `pitch` apart, and that memory."""
    rows, cols = x.shape
    space = torch.full((off + (rows - 1) * pitch + cols,), 7.0, dtype=x.dtype, device="cuda")
    view = space.as_strided((rows, cols), (pitch, 1), storage_offset=off)
    view.copy_(x)
    return view, space


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [1, 5, 8, 40, 257, 771, 1032, 2600])
def test_norm_and_its_gradients_are_the_same_at_every_offset(z, cols, dtype, kept):
    """Every matrix at another offset, ends of rows anywhere in a 16-byte word:
    the bits of the same call on rows that begin on 16 bytes."""
    rows, up = 6, -(-cols // 8) * 8
    x, r, dy, dh = (normal(rows, cols, dtype, k) for k in range(4))
    w = _weight(cols, dtype)
    aligned = lambda t: _laid(t, 0, up)[0]  # noqa: E731
    want = z.rms_norm(aligned(x), w, residual=aligned(r), y8=True, h8=True)
    h = want.h8 if kept else aligned(want.h)
    want_dx, want_dw = z.rms_norm_backward(aligned(dy), h, w, want.rstd, dh=aligned(dh))
    for off in range(8):
        at = [((off + k) % 8, cols + (off * k) % 5) for k in range(4)]
        n = z.rms_norm(_laid(x, *at[0])[0], w, residual=_laid(r, *at[1])[0], y=_laid(x, *at[2])[0], h=_laid(x, *at[3])[0],
                       y8=True, h8=True)
        assert torch.equal(n.y, want.y) and torch.equal(n.h, want.h) and torch.equal(n.rstd, want.rstd)
        assert torch.equal(n.y8.codes, want.y8.codes) and torch.equal(n.h8.codes, want.h8.codes)
        into, space = _laid(x, *at[2])
        dx, dw = z.rms_norm_backward(_laid(dy, *at[0])[0], h if kept else _laid(want.h, *at[1])[0], w, n.rstd,
                                     dh=_laid(dh, *at[3])[0], dx=into)
        assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw), (off, at)
        rest = torch.ones(space.shape[0], dtype=torch.bool, device="cuda")
        rest.as_strided(dx.shape, dx.stride(), storage_offset=at[2][0]).fill_(False)
        assert (space[rest] == 7.0).all()


def test_norm_backward_twice_is_the_same(z):
    h, dy, w = normal(3001, 1000, "bf16", 1), normal(3001, 1000, "bf16", 2), _weight(1000, "bf16")
    rstd = ref.norm(h, w, 1e-6)[1].float()
    a, b = z.rms_norm_backward(dy, h, w, rstd), z.rms_norm_backward(dy, h, w, rstd)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("cols", [64, 300, 512, 1024, 2048, 3000, 4096, 8192, 20000])
def test_a_rows_results_are_the_same_in_every_batch(z, cols):
    """However many rows there are, and with them other blocks and lanes."""
    rows = (1 << 22) // cols + 3
    x, w = normal(rows, cols, "bf16", 11), _weight(cols, "bf16")
    all_rows = z.rms_norm(x, w, y8=True)
    for first, last in ((0, 1), (5, 22), (rows - 40, rows)):
        some = z.rms_norm(x[first:last], w, y8=True)
        assert torch.equal(some.rstd, all_rows.rstd[first:last]) and torch.equal(some.y, all_rows.y[first:last])
        assert torch.equal(some.y8.codes[:, :cols], all_rows.y8.codes[first:last, :cols])
        blocks = -(-cols // 32)  # (what is behind them is nobody's)
        assert torch.equal(some.y8.scales[:, :blocks], all_rows.y8.scales[first:last, :blocks])


@pytest.mark.parametrize("cols,rows", [(1, (1 << 29) + 1003), (72, (1 << 26) + 1003)])
def test_more_rows_than_32_bits_count_lanes_of(z, cols, rows):
    """Rows share blocks: their lanes' number passes 2^32, their elements' too."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("wants 40 GB")
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    w = _weight(cols, "bf16")
    ends = (slice(0, 777), slice(rows - 777, rows))
    for k, e in enumerate(ends):
        x[e] = normal(777, cols, "bf16", 5 + k)
    small = [(x[e].clone(), z.rms_norm(x[e], w)) for e in ends]
    y = torch.empty_like(x)
    n = z.rms_norm(x, w, y=y)
    for e, (_, want) in zip(ends, small):
        assert torch.equal(n.y[e], want.y) and torch.equal(n.rstd[e], want.rstd)
    dx, _ = z.rms_norm_backward(y, x, w, n.rstd, dx=y)  # y as dy, its gradient in its place
    for e, (h, want) in zip(ends, small):
        assert torch.equal(dx[e], z.rms_norm_backward(want.y, h, w, want.rstd)[0])


@pytest.mark.parametrize("cols", [48, 800, 20000])
def test_norm_backward_against_differences(z, cols):
    """Central differences of the 64-bit norm: their own error is of the order
    of step^2 = 1e-10 times a third derivative of about 1."""
    rows, step, eps = 3, 1e-5, 1e-6
    h, w, dy = normal(rows, cols, "f32", 1), _weight(cols, "f32"), normal(rows, cols, "f32", 2)
    n = z.rms_norm(h, w, eps)
    dx, dw = z.rms_norm_backward(dy, h, w, n.rstd)
    loss = lambda h, w: (ref.norm(h, w, eps)[0] * dy.double()).sum()  # noqa: E731
    for i, j in ((0, 0), (1, cols // 2), (2, cols - 1)):
        up, down = h.double(), h.double()
        up[i, j] += step
        down[i, j] -= step
        assert abs(float(loss(up, w) - loss(down, w)) / (2 * step) - float(dx[i, j])) < 2e-5
        up, down = w.double(), w.double()
        up[j] += step
        down[j] -= step
        assert abs(float(loss(h, up) - loss(h, down)) / (2 * step) - float(dw[j])) < 2e-5


def test_norm_backward_keeps_nan_within_rows_and_shows_it_in_dw(z):
    h, dy, w = normal(9, 300, "bf16", 1), normal(9, 300, "bf16", 2), _weight(300, "bf16")
    rstd = ref.norm(h, w, 1e-6)[1].float()
    want, _ = z.rms_norm_backward(dy, h, w, rstd)
    dy[4, 7] = float("nan")
    dx, dw = z.rms_norm_backward(dy, h, w, rstd)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(dx[keep], want[keep]) and torch.isnan(dx[4]).all()
    assert torch.isnan(dw[7]) and torch.isfinite(dw[:7]).all() and torch.isfinite(dw[8:]).all()


def test_norm_without_rows_or_columns(z):
    w = _weight(64, "bf16")
    x = normal(0, 64, "bf16", 1)
    n = z.rms_norm(x, w, residual=x, y8=True)
    assert tuple(n.y.shape) == (0, 64) and tuple(n.rstd.shape) == (0,)
    dw = torch.full((64,), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, _ = z.rms_norm_backward(x, x, w, n.rstd, dw=dw)
    assert not dw.any() and tuple(dx.shape) == (0, 64)
    x = torch.empty(4, 0, dtype=torch.bfloat16, device="cuda")
    assert tuple(z.rms_norm(x, w[:0], rstd=False).y.shape) == (4, 0)


def test_norm_past_32_bit_offsets(z):
    rows, cols = 70001, 1 << 15
    w = _weight(cols, "bf16")
    last = normal(3, cols, "bf16", 3)
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = last
    want = z.rms_norm(last, w, y8=True)
    n = z.rms_norm(x, w, y8=True)
    assert torch.equal(n.y[-3:], want.y) and torch.equal(n.y8.codes[-3:], want.y8.codes)
    dy = torch.zeros_like(x)
    dy[-3:] = last.flip(0)
    dx, dw = z.rms_norm_backward(dy, x, w, n.rstd)
    want_dx, want_dw, off_dx, off_dw = ref.norm_backward(last.flip(0), last, w, want.rstd)
    ref.assert_near(dx[-3:], want_dx, off_dx, "dx")
    ref.assert_near(dw, want_dw, off_dw, "dw")
    assert not dx[:-3].any()


def test_wrappers_refuse_what_does_not_fit(z):
    x, w = normal(8, 64, "bf16", 1), _weight(64, "bf16")
    rstd = torch.ones(8, device="cuda")
    for call in (lambda: z.rms_norm(x, w[:63]), lambda: z.rms_norm(x, w.double()), lambda: z.rms_norm(x, x[:, 0]),
                 lambda: z.rms_norm(x, w, residual=x.float()), lambda: z.rms_norm(x, w, residual=x[:7]),
                 lambda: z.rms_norm(x, w, y=x.half()), lambda: z.rms_norm(x, w, y8=z.mx8_empty(8, 65)),
                 lambda: z.rms_norm(x, w, y8=z.mx4_empty(8, 64)), lambda: z.rms_norm(x, w, rstd=rstd.half()),
                 lambda: z.rms_norm(x.t(), w), lambda: z.rms_norm_backward(x, x.float(), w, rstd),
                 lambda: z.rms_norm_backward(x, x, w, rstd[:7]), lambda: z.rms_norm_backward(x, x, w, rstd.half()),
                 lambda: z.rms_norm_backward(x, z.mx8_empty(7, 64), w, rstd),
                 lambda: z.rms_norm_backward(x, x, w, rstd, dw=w[:63]), lambda: z.rms_norm_backward(x, x, w, rstd, dx=x[:7])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: z.rms_norm(x, w, eps=0.0), lambda: z.rms_norm(x, w, y=False, rstd=False),
                 lambda: z.rms_norm_backward(x[:1].expand(8, 64), x, w, rstd)):
        with pytest.raises(z.ZeroError):
            call()
