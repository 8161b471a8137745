"""GPU tests of the MX4 operators (zero_mx4_*) against plain 64-bit
arithmetic: quantisation and read-back bit for bit, the collectives bit for
bit against the 16-bit ones, the product within its rounding bounds."""
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def _normal(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(rows, cols, generator=g, device="cuda")).to(DTYPES[dtype])


def _assert_mx4(m, code, s, what):
    got_code, got_s = ref.unpack(m)
    assert torch.equal(got_s, s), f"{what}: scales differ"
    assert torch.equal(got_code, code), f"{what}: {int((got_code != code).sum())} codes differ"


def _same_values(got, want, what):
    """Equal 64-bit values, NaN equal to NaN."""
    got, want = got.double(), want.double()
    bad = ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), f"{what}: {int(bad.sum())} values differ"


# ------------------------------------------------------------- quantisation --

SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (5, 64), (1, 255), (7, 257), (33, 100), (128, 64), (129, 65), (200, 513),
          (64, 1024), (300, 768)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", [None, 0, (7 << 40) + 12345])
def test_quantize_rows_columns_and_both(z, dtype, shape, seed):
    x = _normal(*shape, dtype, sum(shape))
    want, want_t = ref.quantize(x, seed), ref.quantize(x.t(), seed)
    _assert_mx4(z.mx4_quantize(x, seed=seed), *want, "rows")
    _assert_mx4(z.mx4_quantize(x, transpose=True, seed=seed), *want_t, "columns")
    a, b = z.mx4_quantize_both(x, seed)
    _assert_mx4(a, *want, "both, rows")
    _assert_mx4(b, *want_t, "both, columns")


def _special(dtype):
    """Rows that meet every rounding tie, the format's ends, empty blocks,
    infinities and NaN."""
    t = DTYPES[dtype]
    fi = torch.finfo(t)
    x = torch.zeros(12, 96, dtype=torch.float64)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.0, 6.0, 7.9, 0.1])
    x[0, :12], x[0, 12:24] = ties, -ties
    x[1, 32:44] = ties / 1024  # with 7.9 / 1024 as the block's largest
    x[2, 40] = fi.max
    x[2, 41] = -fi.max / 3
    x[3, 0] = fi.smallest_normal
    x[3, 1] = fi.tiny / 2  # below the normal numbers
    x[4, 64] = fi.smallest_normal * fi.eps  # the least subnormal
    x[5, 70] = float("inf")
    x[5, 71] = 1.0
    x[6, 5] = float("-inf")
    x[7, 33] = float("nan")
    x[7, 1] = 3.0
    x[8] = -0.0
    x[9, 95] = 1.0
    x[10] = torch.linspace(-8, 8, 96)
    x[11] = 2.0 ** torch.linspace(-20, 15, 96).floor()
    return x.to(t).cuda()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("seed", [None, 3])
def test_quantize_ties_ends_empty_blocks_and_nonfinite(z, dtype, seed):
    x = _special(dtype)
    m, mt = z.mx4_quantize_both(x, seed)
    _assert_mx4(m, *ref.quantize(x, seed), "rows")
    _assert_mx4(mt, *ref.quantize(x.t(), seed), "columns")
    _assert_mx4(z.mx4_quantize(x, seed=seed), *ref.quantize(x, seed), "rows alone")
    # read back: exact in bf16 and binary32, to nearest even in binary16
    for t in DTYPES.values():
        _same_values(z.mx4_dequantize(m, t), ref.read(m).to(t), f"read back as {t}")
    # the transpose of the MX4 matrix: new blocks of its values
    _assert_mx4(z.mx4_transpose(m, seed), *ref.quantize(ref.read(m).float().t(), seed), "transpose")


@pytest.mark.parametrize("ld,off", [(100, 0), (101, 0), (104, 0), (104, 1), (128, 8)])
def test_quantize_strided_source_and_pitched_result(z, ld, off):
    """Rows apart by more than their length, at addresses of every alignment;
    results between guard bytes."""
    rows, cols = 37, 100
    big = _normal(1, rows * ld + off + 8, "bf16", 5).view(-1)
    x = big[off:off + rows * ld].view(rows, ld)[:, :cols]
    codes = torch.full((rows, 96), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 9), 0xA5, dtype=torch.uint8, device="cuda")
    out = z.MX4(codes, scales, rows, cols)
    z.mx4_quantize(x, out=out)
    _assert_mx4(out, *ref.quantize(x), "strided")
    assert (codes[:, 64:] == 0xA5).all() and (scales[:, 4:] == 0xA5).all()
    y = torch.full((rows, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    z.mx4_dequantize(out, out=y[:, :cols])
    _same_values(y[:, :cols], ref.read(out), "read back into a strided matrix")
    assert (y[:, cols:] == 7.0).all()
    codes_t = torch.full((cols, 48), 0xA5, dtype=torch.uint8, device="cuda")
    scales_t = torch.full((cols, 3), 0xA5, dtype=torch.uint8, device="cuda")
    out_t = z.MX4(codes_t, scales_t, cols, rows)
    z.mx4_quantize(x, transpose=True, out=out_t)
    _assert_mx4(out_t, *ref.quantize(x.t()), "strided, columns")
    assert (codes_t[:, 32:] == 0xA5).all() and (scales_t[:, 2:] == 0xA5).all()


@pytest.mark.parametrize("shape", [(1, 1), (40, 33), (129, 200), (257, 96)])
def test_transpose(z, shape):
    m = z.mx4_quantize(_normal(*shape, "bf16", 2, 0.02))
    for seed in (None, 11):
        _assert_mx4(z.mx4_transpose(m, seed), *ref.quantize(ref.read(m).float().t(), seed), "transpose")


def test_stochastic_rounding_has_the_mean(z):
    """The mean over 4096 seeds of a value between two grid points: each draw
    is one of the two, so the mean's deviation is at most step / 2 / 64; seven
    deviations allowed, over 32 elements."""
    x = torch.linspace(0.05, 6.0, 32, device="cuda").view(1, 32)
    total = torch.zeros(1, 32, dtype=torch.float64, device="cuda")
    n = 4096
    for seed in range(n):
        total += z.mx4_dequantize(z.mx4_quantize(x, seed=seed), torch.float32).double()
    step = torch.where(x < 2, 0.5, torch.where(x < 4, 1.0, 2.0)).double()
    assert ((total / n - x.double()).abs() <= step * (7 / (2 * n ** 0.5) + 2.0 ** -16)).all()


# ------------------------------------------------------------------ product --

def _assert_product(got, a, b, what):
    """Elements' products are exact; a 32-bit sum of K terms is off by at most
    2^-23 of the terms' magnitudes' sum for each of its additions (truncating
    ones included), at most K / 32 + 16 of them one after another (blocks,
    then the parts of a split k); the result is rounded once."""
    a, b = ref.read(a), ref.read(b)
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    eps = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -149
    tol = (a.shape[1] / 32 + 16) * 2.0 ** -23 * mag * (1 + eps) + eps * want.abs() + tiny
    bad = ~((got.double() - want).abs() <= tol)
    bad &= ~(got.isnan() & want.isnan())
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst " \
                          f"{float(((got.double() - want).abs() / tol)[~want.isnan()].max()):.3g} times it"


PRODUCTS = [(1, 1, 1), (1, 128, 32), (1, 130, 33), (2, 100, 64), (8, 256, 256), (9, 257, 300), (17, 1000, 771),
            (32, 128, 512), (33, 129, 257), (64, 640, 2048), (100, 200, 4100), (128, 128, 128), (129, 300, 96),
            (256, 256, 1024), (300, 1000, 771), (1000, 333, 100), (2048, 2047, 100), (1999, 1800, 300), (513, 768, 2304), (1, 4096, 4096), (2048, 2304, 768),
            (2500, 2700, 544), (3330, 3200, 300), (3100, 3601, 1040)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(z, m, n, k):
    a = z.mx4_quantize(_normal(m, k, "bf16", m + k))
    b = z.mx4_quantize(_normal(n, k, "bf16", n + k, 0.02))
    for name, t in DTYPES.items():
        got = z.mx4_matmul(a, b, t)
        _assert_product(got, a, b, name)
        assert torch.equal(got, z.mx4_matmul(a, b, t)), "two runs differ"
    z.mx4_check()


@pytest.mark.parametrize("m,n,k", [(1, 128, 256), (7, 300, 800), (130, 520, 416), (600, 700, 288), (2400, 2432, 320)])
def test_matmul_of_whole_numbers_is_exact(z, m, n, k):
    """Every scale 2 and 4 and even elements: all sums are whole numbers below 2^24."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    pick = lambda r: torch.randint(0, 16, (r, ref.blocks_of(k), 32), generator=g, device="cuda")  # noqa: E731
    scale = lambda r: torch.randint(128, 130, (r, ref.blocks_of(k)), generator=g, device="cuda")  # noqa: E731
    a = z.MX4(*ref.pack(pick(m), scale(m)), m, k)
    b = z.MX4(*ref.pack(pick(n), scale(n)), n, k)
    assert torch.equal(z.mx4_matmul(a, b, torch.float32).double(), ref.read(a) @ ref.read(b).t())


@pytest.mark.parametrize("m", [3, 200])
@pytest.mark.parametrize("scale_pitch", [25, 26, 28, 31])
@pytest.mark.parametrize("ld,off", [(300, 0), (301, 0), (304, 0), (304, 3), (320, 16)])
def test_matmul_pitches_and_alignments(z, m, scale_pitch, ld, off):
    """Scale rows and results at every alignment; the bytes past a row's
    blocks hold NaN scales, the elements around the result stay."""
    n, k = 300, 796
    parts = []
    for rows in (m, n):
        code, s = ref.quantize(_normal(rows, k, "f32", rows))
        c, sc = ref.pack(code, s, 416, scale_pitch)
        sc[:, 25:] = 255
        c[:, 400:] = 0x77
        parts.append(z.MX4(c, sc, rows, k))
    a, b = parts
    whole = torch.full((off + m * ld + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = whole[off:off + m * ld].view(m, ld)
    z.mx4_matmul(a, b, out=out[:, :n])
    _assert_product(out[:, :n], a, b, "strided")
    assert (out[:, n:] == 5.0).all() and (whole[:off] == 5.0).all() and (whole[off + m * ld:] == 5.0).all()


@pytest.mark.parametrize("m,n", [(5, 200), (200, 260), (2000, 2600), (3400, 3400)])
def test_matmul_zero_rows_nan_blocks_and_extreme_scales(z, m, n):
    k = 192
    x, y = _normal(m, k, "f32", 1), _normal(n, k, "f32", 2)
    x[m - 1] = 0.0  # a row that a mask emptied
    y[3] = 0.0
    x[0, 40] = float("nan")
    y[n - 1, 191] = float("inf")
    x[1] *= 2.0 ** 100
    y[4] *= 2.0 ** -110
    a, b = z.mx4_quantize(x), z.mx4_quantize(y)
    got = z.mx4_matmul(a, b, torch.float32)
    assert got[0].isnan().all() and got[:, n - 1].isnan().all()
    fine = got[1:, :n - 1]
    assert not fine.isnan().any()
    assert (got[m - 1, :n - 1] == 0).all() and (got[1:, 3] == 0).all()
    _assert_product(got, a, b, "extremes")


@pytest.mark.parametrize("n,k", [(1, 1), (1, 32), (7, 33), (33, 771), (9500, 96), (130, 4128), (300, 2049), (40, 22528),
                                 (40, 22529), (5000, 2080)])
@pytest.mark.parametrize("low,high", [((100, 140), (100, 140)), ((0, 12), (90, 130)), ((0, 12), (244, 255)),
                                      ((244, 255), (0, 12)), ((0, 40), (0, 120))])
def test_matmul_of_one_row(z, n, k, low, high):
    """Scales over their whole range, every code, rows of scales at odd
    offsets, one block in 50 of b NaN; a sum that falls below the normal
    numbers is off by at most half their smallest step for each of a block's
    terms and the lanes' five additions (all terms here stay below 2^128)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n + k)
    nb = ref.blocks_of(k)

    def matrix(rows, scales, nan):
        code = torch.randint(0, 16, (rows, nb, 32), generator=g, device="cuda")
        code[:, -1, k - 32 * (nb - 1):] = 0
        s = torch.randint(*scales, (rows, nb), generator=g, device="cuda")
        if nan:
            s[torch.rand(rows, nb, generator=g, device="cuda") < 1 / (50 * nb)] = 255
        return z.MX4(*ref.pack(code, s, scale_pitch=nb + 1), rows, k)

    a, b = matrix(1, low, False), matrix(n, high, True)
    for t in (torch.float32, torch.bfloat16):
        got = z.mx4_matmul(a, b, t)
        u, v = ref.read(a), ref.read(b)
        want, mag = u @ v.t(), u.abs() @ v.abs().t()
        eps = 0.0 if t == torch.float32 else 2.0 ** -8
        tiny = 2.0 ** -149 * (nb + 6) + (0.0 if t == torch.float32 else 2.0 ** -134)
        tol = (nb / 32 + 7) * 2.0 ** -24 * mag * (1 + eps) + eps * want.abs() + tiny
        fine = (got.double() - want).abs() <= tol
        assert (fine | (got.isnan() & want.isnan())).all()


def test_matmul_of_one_row_beyond_the_result_type(z):
    """Positive elements of a large row: infinite where the type's range ends."""
    one = lambda s: z.MX4(*ref.pack(torch.full((3, 2, 32), 2, device="cuda"), torch.full((3, 2), s, device="cuda")), 3, 64)  # noqa: E731
    row = lambda s: z.MX4(*ref.pack(torch.full((1, 2, 32), 2, device="cuda"), torch.full((1, 2), s, device="cuda")), 1, 64)  # noqa: E731
    assert (z.mx4_matmul(row(254), one(254), torch.float32) == float("inf")).all()
    assert (z.mx4_matmul(row(137), one(127), torch.float16) == float("inf")).all()
    assert (z.mx4_matmul(row(136), one(127), torch.float16) == 32768.0).all()
    assert (z.mx4_matmul(row(0), one(0), torch.float32) == 0).all()


def test_matmul_without_columns_or_rows(z):
    out = torch.full((3, 5), 9.0, device="cuda")
    z.mx4_matmul(z.mx4_empty(3, 0), z.mx4_empty(5, 0), out=out)
    assert (out == 0).all()
    assert z.mx4_matmul(z.mx4_empty(0, 64), z.mx4_empty(5, 64)).shape == (0, 5)
    assert z.mx4_linear(torch.empty(0, 64, device="cuda"), z.mx4_empty(5, 64)).shape == (0, 5)
    assert z.mx4_quantize(torch.empty(0, 64, device="cuda")).rows == 0


# ------------------------------------------------------------------- linear --

LINEAR = [(1, 128, 32), (1, 200, 22528), (1, 200, 22529), (1, 2304, 768), (1, 1000, 771), (3, 300, 256), (16, 640, 512), (16, 300, 779), (5, 200, 2080), (2, 130, 800), (9, 70, 4000), (17, 640, 544), (100, 768, 2304),
          (257, 513, 1000), (1000, 2304, 768), (2300, 2200, 512),
          (3330, 3300, 520), (3101, 3800, 771)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,out,inner", LINEAR)
def test_linear_is_quantize_and_matmul(z, dtype, tokens, out, inner):
    x = _normal(tokens, inner, dtype, tokens)
    x[tokens // 2:] *= 0 if tokens > 4 else 1  # padded tokens
    w = z.mx4_quantize(_normal(out, inner, "bf16", out, 0.02))
    xq = z.mx4_quantize(x)
    y = z.mx4_linear(x, w)
    assert y.dtype == x.dtype and torch.equal(y, z.mx4_matmul(xq, w, x.dtype))
    _assert_product(y, xq, w, "linear")
    # a weight whose scale rows lie end to end, and rows of x apart
    tight = z.MX4(w.codes, w.scales[:, :ref.blocks_of(inner)].contiguous(), out, inner)
    wide = torch.zeros(tokens, inner + 5, dtype=x.dtype, device="cuda")
    wide[:, :inner] = x
    assert torch.equal(z.mx4_linear(wide[:, :inner], tight), y)


@pytest.mark.parametrize("tokens", [1, 7, 16, 40])
def test_linear_of_tokens_that_are_zero_nan_or_infinite(z, tokens):
    """A token's block that is not finite makes that token's outputs NaN and
    no other's; an empty token's outputs are zero."""
    x = _normal(tokens, 800, "bf16", 1)
    x[0, 300] = float("nan") if tokens % 2 else float("-inf")
    x[tokens - 1, :] = 0.0 if tokens > 1 else x[0]
    w = z.mx4_quantize(_normal(200, 800, "bf16", 2))
    y = z.mx4_linear(x, w)
    assert y[0].isnan().all() and not y[1:].isnan().any()
    if tokens > 1:
        assert (y[-1] == 0).all()
    _assert_product(y, z.mx4_quantize(x), w, "linear")


def test_matrices_past_32_bit_offsets(z):
    """4.6e9 elements: the ends of rows and of the matrix, quantised along the
    rows and down the columns, read back, and as a product's result."""
    rows, cols = 70016, 65600
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, 32768, 65535, 65536, rows - 33, rows - 1]
    for i in at:
        x[i] = _normal(1, cols, "bf16", i)[0]
    m = z.mx4_quantize(x)
    for i in at:
        one = z.MX4(m.codes[i:i + 1], m.scales[i:i + 1], 1, cols)
        _assert_mx4(one, *ref.quantize(x[i:i + 1]), f"row {i}")
    back = z.mx4_dequantize(m)
    for i in at:
        _same_values(back[i:i + 1], ref.rounded(x[i:i + 1]), f"row {i} read back")
    assert (back[2:100] == 0).all() and (back[rows - 32:rows - 1] == 0).all()
    del m, back
    t = z.mx4_quantize(x, transpose=True)
    for j in (0, 40000, cols - 1):
        one = z.MX4(t.codes[j:j + 1], t.scales[j:j + 1], 1, rows)
        _assert_mx4(one, *ref.quantize(x[:, j:j + 1].t().contiguous()), f"column {j}")
    del t, x
    a, b = z.mx4_quantize(_normal(rows, 64, "bf16", 1)), z.mx4_quantize(_normal(cols, 64, "bf16", 2))
    y = z.mx4_matmul(a, b)
    pick = lambda m, i: z.MX4(m.codes[i:i + 40], m.scales[i:i + 40], 40, 64)  # noqa: E731
    for i in (0, 65520, rows - 40):
        for j in (0, 65500, cols - 40):
            _assert_product(y[i:i + 40, j:j + 40], pick(a, i), pick(b, j), f"rows {i}, columns {j}")


def test_linear_wants_no_more_than_its_workspace(z):
    """The bytes around the workspace, the operands and the result stay."""
    import ctypes

    for tokens, out, inner, pitch in ((1, 300, 771, 25), (40, 300, 768, 24), (700, 2600, 800, 25), (1, 256, 512, 16),
                                      (3300, 3300, 96, 3), (3300, 3300, 600, 32)):
        x = _normal(tokens, inner, "bf16", 3)
        c, s = ref.pack(*ref.quantize(_normal(out, inner, "f32", 4, 0.02)), scale_pitch=pitch)
        w = z.MX4(c, s, out, inner)
        need = ctypes.c_int64()
        assert z.zero_mx4_linear_workspace(tokens, w._c, need) == 0
        space = torch.full((need.value + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        y = torch.full((tokens + 2, out), 3.0, dtype=torch.bfloat16, device="cuda")
        at = space.data_ptr() + 256
        args = (x.data_ptr(), z.ZERO_DTYPE_BF16, tokens, inner, w._c, y[1:].data_ptr(), z.ZERO_DTYPE_BF16, out, at)
        stream = torch.cuda.current_stream().cuda_stream
        if need.value:
            assert z.zero_mx4_linear(*args, need.value - 1, stream) == z.ZERO_EINVAL
            assert z.zero_mx4_linear(*args[:-1], None, need.value, stream) == z.ZERO_EINVAL
            assert z.zero_mx4_linear(*args[:-1], at + 8, need.value, stream) == z.ZERO_EINVAL
        assert z.zero_mx4_linear(*args, need.value, stream) == 0
        assert torch.equal(y[1:-1], z.mx4_linear(x, w))
        assert (y[0] == 3).all() and (y[-1] == 3).all()
        assert (space[:256] == 0xA5).all() and (space[256 + need.value:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,out,inner", [(1, 64, 32), (33, 100, 77), (300, 768, 256), (1003, 520, 384),
                                              (3330, 300, 3200), (300, 3330, 3201), (3100, 3400, 3600)])
@pytest.mark.parametrize("seed", [None, 12345])
def test_linear_backward(z, dtype, tokens, out, inner, seed):
    x, dy = _normal(tokens, inner, dtype, 1), _normal(tokens, out, dtype, 2, 0.25)
    w = z.mx4_quantize(_normal(out, inner, "bf16", 3, 0.02))
    dx, dw = z.mx4_linear_backward(dy, x, w, seed=seed)
    dyq, dyq_t = z.mx4_quantize_both(dy, seed)
    _assert_mx4(dyq, *ref.quantize(dy, seed), "dy")
    _assert_mx4(dyq_t, *ref.quantize(dy.t(), seed), "dy^T")
    _assert_product(dx, dyq, z.mx4_transpose(w), "dx")
    _assert_product(dw, dyq_t, z.mx4_quantize(x, transpose=True), "dw")
    assert dx.shape == x.shape and dw.shape == (out, inner)


def test_linear_backward_strides_types_and_empty_batches(z):
    """Mixed types, rows apart, gradients into views (guarded), no tokens, no
    outputs."""
    t, o, k = 70, 96, 160
    x, dy = _normal(t, k + 3, "f32", 1)[:, :k], _normal(t, o + 8, "bf16", 2)[:, 8:]
    w = z.mx4_quantize(_normal(o, k, "bf16", 3, 0.02))
    dxs = torch.full((t, k + 4), 3.0, dtype=torch.float16, device="cuda")
    flat = torch.full((o * k + 16,), 3.0, dtype=torch.bfloat16, device="cuda")  # a rank's gradient buffer
    dx, dw = z.mx4_linear_backward(dy, x, w, dx=dxs[:, :k], dw=flat[8:-8].view(o, k))
    _assert_product(dx, z.mx4_quantize(dy), z.mx4_transpose(w), "dx")
    _assert_product(dw, z.mx4_quantize(dy, transpose=True), z.mx4_quantize(x, transpose=True), "dw")
    assert (dxs[:, k:] == 3).all() and (flat[:8] == 3).all() and (flat[-8:] == 3).all()
    dx, dw = z.mx4_linear_backward(dy[:0], x[:0], w, dw=flat[8:-8].view(o, k))
    assert dx.shape == (0, k) and (dw == 0).all()
    dx, dw = z.mx4_linear_backward(dy[:, :0], x, z.mx4_empty(0, k))
    assert (dx == 0).all() and dx.shape == (t, k) and dw.shape == (0, k)


def test_linear_backward_against_differences(z):
    """On inputs that every quantisation keeps exactly -- whole numbers of
    magnitude 4 or 6 or 0, one of them in each block along either axis, so
    that every block's scale is 1 -- y is linear in x and in w, and its
    differences are the gradients, exactly."""
    t, o, k = 64, 96, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def pick(rows, cols):
        v = torch.tensor([4.0, -4.0, 6.0, -6.0], device="cuda")
        return v[torch.randint(0, 4, (rows, cols), generator=g, device="cuda")]

    x, wv, dy = pick(t, k), pick(o, k), pick(t, o)
    w = z.mx4_quantize(wv)
    dx, dw = z.mx4_linear_backward(dy, x, w, dx=torch.empty(t, k, device="cuda"), dw=torch.empty(o, k, device="cuda"))
    loss = lambda x, w: (z.mx4_linear(x, w).double() * dy.double()).sum()  # noqa: E731
    for i, j in ((0, 0), (5, 77), (63, 127)):
        moved = x.clone()
        moved[i, j] = -moved[i, j]
        assert float(loss(moved, w) - loss(x, w)) == float((moved - x)[i, j] * dx[i, j])
    for i, j in ((0, 0), (50, 3), (95, 127)):
        moved = wv.clone()
        moved[i, j] = -moved[i, j]
        assert float(loss(x, z.mx4_quantize(moved)) - loss(x, w)) == float((moved - wv)[i, j] * dw[i, j])


# -------------------------------------------------------------- collectives --

def _context(z, stage, n_ranks, numel, dtype="bf16", seed=0, **kw):
    opt = z.ZeroOptimizer([n for n, _ in numel], [layer for _, layer in numel], n_ranks, stage,
                          dtype=z.ZERO_DTYPE_F16 if dtype == "f16" else z.ZERO_DTYPE_BF16, **kw)
    master = opt.view(z.ZERO_VIEW_MASTER)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    master.copy_(0.02 * torch.randn(opt.psi_pad, generator=g, device="cuda"))
    opt.load_master()
    return opt


@pytest.mark.parametrize("stage", [1, 2, 3])
@pytest.mark.parametrize("n_ranks", [1, 3, 8, 11])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_all_gather_quantises_the_owners_parameters(z, stage, n_ranks, dtype):
    """Every rank's buffers, every shard boundary, a ragged last block, guard
    bytes after each buffer; the replicas of stages 1 and 2 differ here, so
    that only the owner's copy gives the right answer."""
    opt = _context(z, stage, n_ranks, [(1000, 0), (333, 0), (4100, 1)], dtype)
    S = opt.shard
    if stage == 3:
        flat = opt.view(z.ZERO_VIEW_PARAM).view(DTYPES[dtype])
    else:
        for r in range(n_ranks):
            own = opt.view(z.ZERO_VIEW_PARAM, r).view(DTYPES[dtype])
            own[:r * S] = 9.0
            own[(r + 1) * S:] = 9.0
        flat = torch.cat([opt.view(z.ZERO_VIEW_PARAM, r).view(DTYPES[dtype])[r * S:(r + 1) * S] for r in range(n_ranks)])
    for lo, hi in ((0, opt.psi_pad), (8, 8), (8, 16), (1000, 1336), (16, opt.psi_pad - 8)):
        nb = ref.blocks_of(hi - lo)
        codes = torch.full((n_ranks, 16 * nb + 64), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((n_ranks, nb + 64), 0xA5, dtype=torch.uint8, device="cuda")
        opt.all_gather_mx4(lo, hi, codes, scales)
        if hi == lo:
            assert (codes == 0xA5).all()
            continue
        want = ref.quantize(flat[lo:hi].view(1, -1))
        for r in range(n_ranks):
            m = z.MX4(codes[r, :16 * nb].view(1, -1), scales[r, :nb].view(1, -1), 1, hi - lo)
            _assert_mx4(m, *want, f"rank {r} of [{lo}, {hi})")
        assert (codes[:, 16 * nb:] == 0xA5).all() and (scales[:, nb:] == 0xA5).all()
    opt.close()


@pytest.mark.parametrize("stage", [2, 3])
@pytest.mark.parametrize("n_ranks", [1, 2, 8, 9, 16, 19])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_reduce_scatter_gives_the_bits_of_the_16_bit_one(z, stage, n_ranks, dtype):
    """The same shard, norm and non-finite count as zero_reduce_scatter of the
    gradients read back (exact in bf16; in binary16 for values of this size).
    The norm's partial sums are added in another order."""
    opt = _context(z, stage, n_ranks, [(4096 + 8 * 37, 0)], dtype, grad_buffers=False)
    lo, hi = 16, opt.psi_pad - 8
    nb = ref.blocks_of(hi - lo)
    codes = torch.empty(n_ranks, 16 * nb, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_ranks, nb, dtype=torch.uint8, device="cuda")
    dense = torch.zeros(n_ranks, hi - lo, dtype=DTYPES[dtype], device="cuda")
    for r in range(n_ranks):
        x = _normal(1, hi - lo, "f32", 100 + r, 2.0 ** (r % 5))
        x[0, 64:96] = 0.0
        if r == n_ranks - 1:
            x[0, 200] = float("nan")
        m = z.MX4(codes[r].view(1, -1), scales[r].view(1, -1), 1, hi - lo)
        z.mx4_quantize(x, seed=r, out=m)
        z.mx4_dequantize(m, out=dense[r].view(1, -1))
    shard = opt.view(z.ZERO_VIEW_GRAD_SHARD)
    shard.fill_(77)
    opt.reduce_scatter_mx4(lo, hi, codes, scales)
    got, stats = shard.clone(), opt.read_stats()
    shard.fill_(77)
    opt.load_master()
    shard.fill_(77)
    opt.reduce_scatter(lo, hi, [d.data_ptr() for d in dense])
    want = opt.read_stats()
    a, b = got.view(DTYPES[dtype]), shard.view(DTYPES[dtype])
    assert torch.equal(torch.where(a.isnan(), 0, got), torch.where(b.isnan(), 0, shard))
    assert torch.equal(a.isnan(), b.isnan()) and int(a[lo:hi].isnan().sum()) == 32
    assert (got[:lo] == 77).all() and (got[hi:] == 77).all()
    assert stats["nonfinite"] == want["nonfinite"] == 32
    opt.close()


@pytest.mark.parametrize("top", [1, 130, 239, 240, 241, 252, 254])
def test_reduce_scatter_over_the_whole_range_of_scales(z, top):
    """Scales from the least to the greatest, in bf16's own range; sums that
    overflow become infinite as the 16-bit sum's do."""
    n, n_ranks = 1024, 3
    opt = _context(z, 2, n_ranks, [(n, 0)], grad_buffers=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(top)
    code = torch.randint(0, 16, (n_ranks, n // 32, 32), generator=g, device="cuda")
    s = torch.randint(max(0, top - 3), top + 1, (n_ranks, n // 32), generator=g, device="cuda")
    codes, scales = ref.pack(code, s)
    dense = ref.values(code, s, n).to(torch.bfloat16).contiguous()
    opt.reduce_scatter_mx4(0, n, codes, scales)
    got = opt.view(z.ZERO_VIEW_GRAD_SHARD)[:n].clone()
    opt.reduce_scatter(0, n, [d.data_ptr() for d in dense])
    want = opt.view(z.ZERO_VIEW_GRAD_SHARD)[:n]
    a, b = got.view(torch.bfloat16), want.view(torch.bfloat16)
    assert torch.equal(a.isnan(), b.isnan())
    assert torch.equal(torch.where(a.isnan(), 0, got), torch.where(b.isnan(), 0, want))
    opt.close()


@pytest.mark.parametrize("n_ranks", [1, 2, 3, 4, 5, 8, 9, 16, 19])
@pytest.mark.parametrize("spread", [0, 3, 4, 5, 9, 40])
def test_reduce_scatter_of_ranks_with_scales_apart(z, n_ranks, spread):
    """Blocks whose scales differ between the ranks by up to `spread` steps and
    by exactly that, largest elements of one sign and of both, against the
    16-bit reduce-scatter of the same values, bit for bit."""
    n, low = 2048, 100
    opt = _context(z, 2, n_ranks, [(n, 0)], grad_buffers=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(100 * n_ranks + spread)
    code = torch.randint(0, 16, (n_ranks, n // 32, 32), generator=g, device="cuda")
    s = low + torch.randint(0, spread + 1, (n_ranks, n // 32), generator=g, device="cuda")
    s[0, :32] = low  # the ends of the spread, at either end of the ranks
    s[n_ranks - 1, 1:32] = low + spread
    s[1:, :4], code[:, :2] = low + spread, 7  # 6 from every rank: the largest sum
    code[:, 2:4] = 15
    code[0, 4:6], s[1:, 4:6], code[1:, 4:6] = 1, low + spread, 7  # and a half beside it
    code[:, 6], s[0, 6] = 0, 0  # rank 0's block empty
    codes, scales = ref.pack(code, s)
    dense = ref.values(code, s, n).to(torch.bfloat16).contiguous()
    opt.reduce_scatter_mx4(0, n, codes, scales)
    got, stats = opt.view(z.ZERO_VIEW_GRAD_SHARD)[:n].clone(), opt.read_stats()
    opt.reduce_scatter(0, n, [d.data_ptr() for d in dense])
    assert torch.equal(got, opt.view(z.ZERO_VIEW_GRAD_SHARD)[:n])
    want = float(got.view(torch.bfloat16).double().square().sum()) ** 0.5
    assert abs(stats["grad_norm"] - want) <= 1e-12 * want and stats["nonfinite"] == 0
    opt.close()


def test_collectives_norm_is_the_sum_over_intervals(z):
    """Two intervals of one step add up; the norm is that of the stored means."""
    opt = _context(z, 2, 4, [(8192, 0)], grad_buffers=False)
    total = 0.0
    for lo, hi in ((0, 4096), (4096, 8192)):
        codes, scales = [], []
        for r in range(4):
            m = z.mx4_quantize(_normal(1, hi - lo, "f32", r + lo, 0.01))
            codes.append(m.codes.reshape(-1).contiguous())
            scales.append(m.scales[0, :128].contiguous())
        opt.reduce_scatter_mx4(lo, hi, codes, scales)
        total += float(opt.view(z.ZERO_VIEW_GRAD_SHARD)[lo:hi].view(torch.bfloat16).double().square().sum())
    assert abs(opt.read_stats()["grad_norm"] - total ** 0.5) <= 1e-12 * total ** 0.5
    opt.close()


def test_collectives_refuse(z):
    opt = _context(z, 2, 2, [(4096, 0)])
    good_c, good_s = torch.empty(2, 2048, dtype=torch.uint8, device="cuda"), torch.empty(2, 128, dtype=torch.uint8, device="cuda")
    for call in (opt.all_gather_mx4, opt.reduce_scatter_mx4):
        for lo, hi in ((4, 64), (0, 4), (0, 8192), (-8, 8), (64, 32)):
            with pytest.raises((z.ZeroError, ValueError)):
                call(lo, hi, good_c, good_s)
        with pytest.raises(ValueError, match="buffers for 2 ranks"):
            call(0, 4096, good_c[:1], good_s[:1])
        with pytest.raises(ValueError, match="bytes a rank"):
            call(0, 4096, good_c[:, :1024].contiguous(), good_s)
        with pytest.raises(ValueError, match="contiguous"):
            call(0, 32, good_c[:, ::2], good_s)
        with pytest.raises(ValueError, match="uint8"):
            call(0, 4096, good_c.view(torch.int8), good_s)
        with pytest.raises(z.ZeroError, match="16-byte"):
            call(0, 32, [good_c[0, 8:], good_c[1]], [good_s[0], good_s[1]])
    opt.close()
    opt = _context(z, 1, 2, [(4096, 0)])
    with pytest.raises(z.ZeroError, match="stage 1"):
        opt.reduce_scatter_mx4(0, 4096, good_c, good_s)
    opt.close()
    opt = _context(z, 2, 2, [(4096, 0)], keep_grad_shards=False)
    with pytest.raises(z.ZeroError, match="dropped"):
        opt.reduce_scatter_mx4(0, 4096, good_c, good_s)
    opt.close()


# ------------------------------------------------- streams, graphs, devices --

def test_captured_and_replayed(z):
    """A captured linear layer forward and backward, replayed on new inputs,
    beside a second graph and eager calls."""
    t, o, k = 200, 2304, 768
    w = z.mx4_quantize(_normal(o, k, "bf16", 1, 0.02))
    tight = z.MX4(w.codes, w.scales[:, :24].contiguous(), o, k)
    x, dy = _normal(t, k, "bf16", 2), _normal(t, o, "bf16", 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z.mx4_linear(x, tight), z.mx4_linear_backward(dy, x, tight)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for weight in (w, tight):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = z.mx4_linear(x, weight)
            one = z.mx4_linear(x[:1], weight)
            dx, dw = z.mx4_linear_backward(dy, x, weight)
        graphs.append((g, y, one, dx, dw))
    for seed in (5, 6, 7):
        x.copy_(_normal(t, k, "bf16", seed))
        dy.copy_(_normal(t, o, "bf16", seed + 50))
        want = (z.mx4_linear(x, w), z.mx4_linear(x[:1], w), *z.mx4_linear_backward(dy, x, w))
        for g, *outs in graphs:
            g.replay()
        for _, *outs in graphs:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_two_streams_at_once_and_a_stream_argument(z):
    """Products of many shapes on two streams side by side, each given its
    stream explicitly while another one is current."""
    shapes = [(1, 2304, 768), (100, 1000, 771), (1000, 2304, 768), (16, 4096, 512)]
    ws = [z.mx4_quantize(_normal(o, k, "bf16", o, 0.02)) for _, o, k in shapes]
    xs = [_normal(t, k, "bf16", t) for t, _, k in shapes]
    want = [z.mx4_linear(x, w) for x, w in zip(xs, ws)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i] = [z.mx4_linear(x, w, stream=s) for x, w in zip(xs, ws)]
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want):
            assert torch.equal(a, b)


def test_linear_right_after_its_operands_are_written(z):
    """The product's early loads of w must not run ahead of the work that
    writes w: all-gather and product in one stream, new parameters each time."""
    o, k, n_ranks = 2304, 768, 4
    opt = _context(z, 3, n_ranks, [(o * k, 0)], seed=3)
    x = _normal(1, k, "bf16", 1)
    codes = torch.zeros(n_ranks, o, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n_ranks, o, k // 32, dtype=torch.uint8, device="cuda")
    params = opt.view(z.ZERO_VIEW_PARAM)
    news = [_normal(1, o * k, "bf16", 20 + i, 0.02)[0] for i in range(6)]
    got = []
    for p in news:
        params[:o * k].view(torch.bfloat16).copy_(p)
        opt.all_gather_mx4(0, o * k, codes, scales)
        got.append([z.mx4_linear(x, z.MX4(c, s, o, k)) for c, s in zip(codes, scales)])
    for p, ys in zip(news, got):
        want = z.mx4_linear(x, z.mx4_quantize(p.view(o, k)))
        for y in ys:
            assert torch.equal(y, want)
    opt.close()


def test_wrappers_refuse_what_does_not_fit(z):
    w = z.mx4_empty(64, 96)
    with pytest.raises(ValueError, match="inputs"):
        z.mx4_linear(torch.zeros(3, 64, device="cuda"), w)
    with pytest.raises(ValueError, match="out is"):
        z.mx4_linear(torch.zeros(3, 96, device="cuda"), w, out=torch.zeros(3, 65, device="cuda"))
    with pytest.raises(ValueError, match="needed"):
        z.mx4_quantize(torch.zeros(3, 96, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError, match="contiguous"):
        z.mx4_quantize(torch.zeros(96, 3, device="cuda").t())
    with pytest.raises(ValueError, match="CUDA matrix"):
        z.mx4_quantize(torch.zeros(96, device="cuda"))
    with pytest.raises(ValueError, match="out is"):
        z.mx4_quantize(torch.zeros(3, 96, device="cuda"), out=w)
    with pytest.raises(z.ZeroError, match="columns"):
        z.mx4_matmul(w, z.mx4_empty(64, 128))
    with pytest.raises(ValueError, match="fit"):
        z.mx4_linear_backward(torch.zeros(3, 60, device="cuda"), torch.zeros(3, 96, device="cuda"), w)


# --------------------------------------------------------- all of them together --

def test_a_training_step_in_four_bits(z):
    """ZeRO-3 training steps of one linear layer over four ranks: the layer is
    gathered in MX4, each rank's forward and backward read it, the gradients
    go out stochastically rounded, are reduce-scattered from MX4 and applied.
    Every part against plain arithmetic on the library's own inputs to it."""
    n_ranks, t, o, k = 4, 96, 256, 512
    opt = _context(z, 3, n_ranks, [(o * k, 0)], seed=11, grad_buffers=False)
    codes = torch.empty(n_ranks, o, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_ranks, o, k // 32, dtype=torch.uint8, device="cuda")
    gcodes, gscales = torch.empty_like(codes), torch.empty_like(scales)
    target = 0.02 * torch.randn(o, k, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    for step in range(1, 4):
        opt.all_gather_mx4(0, o * k, codes, scales)
        params = opt.view(z.ZERO_VIEW_PARAM)[:o * k].view(torch.bfloat16).view(o, k)
        sent = torch.zeros(o, k, device="cuda")  # binary32, in rank order
        for r in range(n_ranks):
            w = z.MX4(codes[r], scales[r], o, k)
            _assert_mx4(w, *ref.quantize(params), "gathered layer")
            x = _normal(t, k, "bf16", 10 * step + r)
            y = z.mx4_linear(x, w)
            _assert_product(y, z.mx4_quantize(x), w, "forward")
            dy = ((y.float() - x.float() @ target.t()) / t).to(torch.bfloat16)
            dx, dw = z.mx4_linear_backward(dy, x, w, seed=step)
            assert dx.shape == x.shape and torch.isfinite(dx).all()
            g = z.MX4(gcodes[r], gscales[r], o, k)
            z.mx4_quantize(dw, seed=1000 * step + r, out=g)
            _assert_mx4(g, *ref.quantize(dw, 1000 * step + r), "sent gradient")
            sent = sent + ref.read(g).float()
        opt.reduce_scatter_mx4(0, o * k, gcodes, gscales)
        shard = opt.view(z.ZERO_VIEW_GRAD_SHARD)[:o * k].view(torch.bfloat16).view(o, k)
        assert torch.equal(shard, (sent * 0.25).to(torch.bfloat16))
        before = opt.view(z.ZERO_VIEW_MASTER).clone()
        opt.adam_shard(-1)
        assert opt.t == step and not torch.equal(before, opt.view(z.ZERO_VIEW_MASTER))
    opt.close()
    z.mx4_check()
