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
            (2500, 2700, 544)]


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


@pytest.mark.parametrize("m,n", [(5, 200), (200, 260), (2000, 2600)])
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


def test_matmul_without_columns_or_rows(z):
    out = torch.full((3, 5), 9.0, device="cuda")
    z.mx4_matmul(z.mx4_empty(3, 0), z.mx4_empty(5, 0), out=out)
    assert (out == 0).all()
    assert z.mx4_matmul(z.mx4_empty(0, 64), z.mx4_empty(5, 64)).shape == (0, 5)
    assert z.mx4_linear(torch.empty(0, 64, device="cuda"), z.mx4_empty(5, 64)).shape == (0, 5)
    assert z.mx4_quantize(torch.empty(0, 64, device="cuda")).rows == 0
