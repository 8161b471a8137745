"""GPU tests of 8-bit checkpoints: quantising and read-back bit for bit against
64-bit arithmetic, and the backward pass of a linear layer from one."""
import pytest
import torch

import layer_reference as ref
from test_gpu_mx4 import _assert_product as assert_product

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def normal(rows, cols, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(rows, cols, generator=g, device="cuda")).to(DTYPES[dtype])


def assert_mx8(m, x, what):
    codes, scales = ref.quantize8(x)
    nb = scales.shape[1]
    assert torch.equal(m.scales[:, :nb].long(), scales), f"{what}: scales"
    assert torch.equal(m.codes[:, :32 * nb].long(), codes), f"{what}: codes"


def same_values(got, want, what):
    """Equal numbers, zeros of equal sign, NaN in the same places."""
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what
    assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, want)), what
    assert torch.equal(torch.signbit(got) & ~nan, torch.signbit(want) & ~nan), what


def read_back(m, dtype):
    """What zero_mx8_dequantize has to give of a matrix that was quantised."""
    v = ref.values8(m.codes, m.scales[:, :-(-m.cols // 32)], m.cols)
    if dtype == torch.float16:
        v = torch.where(torch.isfinite(v), v.clamp(-65504, 65504), v)
    return v.float().to(dtype)


SHAPES = [(1, 1), (1, 32), (3, 33), (5, 255), (7, 256), (2, 257), (1, 4097), (64, 768), (130, 771), (33, 2048), (300, 40),
          (1000, 31)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_and_read_back(z, dtype, shape):
    x = normal(*shape, dtype, 11 * shape[1] + shape[0])
    x[shape[0] // 2:, shape[1] // 2] *= 100
    m = z.mx8_quantize(x)
    assert_mx8(m, x, "quantize")
    for out in DTYPES.values():
        same_values(z.mx8_dequantize(m, out), read_back(m, out), f"read back in {out}")
    assert z.mx8_dequantize(m).dtype == torch.bfloat16


def special(dtype):
    """Blocks at the ends of the range, with ties, of zeros, and not finite."""
    t = DTYPES[dtype]
    info = torch.finfo(t)
    rows = [torch.zeros(32, dtype=torch.float64)]
    rows.append(torch.full((32,), -0.0, dtype=torch.float64))
    grid = torch.tensor(ref.grid8(), dtype=torch.float64)
    ties = (grid[1:] + grid[:-1]) / 2
    for k in range(0, 126, 31):  # ties under the scale of 448, both signs
        rows.append(torch.cat([ties[k:k + 31][:31], torch.tensor([448.0])])[:32])
        rows[-1] = torch.nn.functional.pad(rows[-1], (0, 32 - len(rows[-1])))
        rows.append(-rows[-1])
    for top in (447.9, 448.0, 449.0, 464.0, 479.0, 480.0, 511.0, 512.0, 1.0, 0.4375, 0.438):  # where the scale changes
        rows.append(torch.linspace(-1, 1, 32, dtype=torch.float64) * top)
    for top in (info.max, info.smallest_normal, info.smallest_normal * info.eps, info.max / 3):
        rows.append(torch.linspace(-1, 1, 32, dtype=torch.float64) * float(top))
        rows.append(torch.full((32,), float(top), dtype=torch.float64))
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.linspace(-3, 3, 32, dtype=torch.float64)
        r[17] = bad
        rows.append(r)
        rows.append(torch.linspace(-3, 3, 32, dtype=torch.float64))  # a neighbour that stays as it is
    return torch.stack(rows).to(t).cuda()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_ends_ties_empty_blocks_and_nonfinite(z, dtype):
    x = special(dtype)
    for y in (x, x.reshape(1, -1), x.reshape(1, -1)[:, :-7]):
        m = z.mx8_quantize(y.contiguous())
        assert_mx8(m, y, "special")
        for out in DTYPES.values():
            same_values(z.mx8_dequantize(m, out), read_back(m, out), f"special in {out}")


def test_scales_that_quantising_never_gives(z):
    """0, 1, 2 and 247 .. 254: binary32 holds what it can, bf16 rounds it."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(256, 1).view(256, 256)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1).repeat(1, 8).contiguous()
    m = z.MX8(codes, scales, 256, 256)
    want = ref.values8(codes, scales, 256).float()
    same_values(z.mx8_dequantize(m, torch.float32), want, "every code and scale")
    same_values(z.mx8_dequantize(m), want.bfloat16(), "every code and scale in bf16")


@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("pitch", [320, 301, 304])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strides_alignments_and_pitches(z, dtype, pitch, off):
    """Rows apart, starting off a vector's boundary, into a result whose rows
    are apart: what lies between them stays."""
    rows, cols = 9, 290
    space = normal(rows + 1, pitch, dtype, 5).flatten()
    x = space[off:off + rows * pitch].view(rows, pitch)[:, :cols]
    codes = torch.full((rows, 352), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 13), 0x55, dtype=torch.uint8, device="cuda")
    m = z.MX8(codes, scales, rows, cols)
    assert z.mx8_quantize(x, out=m) is m
    assert_mx8(m, x, "pitched")
    assert (codes[:, 320:] == 0x55).all() and (scales[:, 10:] == 0x55).all()
    back = torch.full((rows * pitch + 9,), 7.0, dtype=DTYPES[dtype], device="cuda")
    out = back[off:off + rows * pitch].view(rows, pitch)[:, :cols]
    z.mx8_dequantize(m, out=out)
    same_values(out, read_back(m, DTYPES[dtype]), "pitched back")
    rest = torch.ones_like(back, dtype=torch.bool)
    rest[off:off + rows * pitch].view(rows, pitch)[:, :cols] = False
    assert (back[rest] == 7.0).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_every_offset_and_many_lengths(z, dtype):
    """Rows that begin and end anywhere in a 16-byte word, of less than a word to
    several warps': the last row's last word is the last of its memory."""
    rows, each = 3, 16 // torch.empty(0, dtype=DTYPES[dtype]).element_size()
    for cols in [*range(1, 26), 31, 32, 33, 64, 65, *range(248, 266), 511, 513, 1023, 1025, 1030]:
        for off in range(each):
            for pitch in (cols, cols + 1, cols + 3):
                n = off + (rows - 1) * pitch + cols
                space = normal(1, n, dtype, cols)[0]
                x = space[off:].as_strided((rows, cols), (pitch, 1), storage_offset=off)
                m = z.mx8_quantize(x)
                back = torch.full((n,), 7.0, dtype=DTYPES[dtype], device="cuda")
                out = back.as_strided((rows, cols), (pitch, 1), storage_offset=off)
                z.mx8_dequantize(m, out=out)
                want = z.mx8_quantize(x.contiguous())
                assert torch.equal(m.codes[:, :cols], want.codes[:, :cols]), (cols, off, pitch)
                flat = torch.empty(rows, cols + 8 - cols % 8, dtype=DTYPES[dtype], device="cuda")[:, :cols]
                assert torch.equal(out, z.mx8_dequantize(want, out=flat)), (cols, off, pitch)
                rest = torch.ones(n, dtype=torch.bool, device="cuda")
                rest.as_strided((rows, cols), (pitch, 1), storage_offset=off).fill_(False)
                assert (back[rest] == 7.0).all(), (cols, off, pitch)


def test_empty(z):
    for shape in ((0, 64), (4, 0)):
        x = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
        m = z.mx8_quantize(x)
        assert tuple(z.mx8_dequantize(m).shape) == shape


def test_past_32_bit_offsets(z):
    rows, cols = 70001, 1 << 16
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    last = normal(3, cols, "bf16", 3)
    x[-3:] = last
    m = z.mx8_quantize(x)
    torch.cuda.synchronize()
    assert_mx8(z.MX8(m.codes[-3:], m.scales[-3:], 3, cols), last, "the last rows")
    assert not m.codes[:-3].any() and (m.scales[:-3] == 3).all()
    x.fill_(1.0)
    z.mx8_dequantize(m, out=x)
    same_values(x[-3:], read_back(z.MX8(m.codes[-3:], m.scales[-3:], 3, cols), torch.bfloat16), "the last rows")
    assert not x[:-3].any()


# ------------------------------------------- a linear layer from a checkpoint --

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,out,inner,seed", [(1, 32, 32, None), (17, 100, 71, None), (128, 256, 512, 3), (333, 1000, 771, 9),
                                                   (1003, 96, 2048, None), (64, 2304, 768, 1)])
def test_linear_backward_from_a_checkpoint(z, dtype, tokens, out, inner, seed):
    """The bits of the same call on the checkpoint's values."""
    dy, w = normal(tokens, out, dtype, 1, 1e-2), z.mx4_quantize(normal(out, inner, "bf16", 2, 0.02))
    kept = z.mx8_quantize(normal(tokens, inner, dtype, 3))
    dx, dw = z.mx4_linear_backward(dy, kept, w, seed=seed)
    assert dx.dtype == dw.dtype == dy.dtype
    x = z.mx8_dequantize(kept)
    want_dx, want_dw = z.mx4_linear_backward(dy, x, w, seed=seed, dx=torch.empty_like(dx))
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
    assert_product(dx, z.mx4_quantize(dy, seed=seed), z.mx4_transpose(w), "dx")
    assert_product(dw, z.mx4_quantize(dy, transpose=True, seed=seed), z.mx4_quantize(x, transpose=True), "dw")


def test_linear_backward_from_a_checkpoint_into_given_results(z):
    """Pitched checkpoint, results of other types, views of a gradient buffer."""
    t, o, k = 40, 96, 160
    dy, w = normal(t, o, "f32", 1, 1e-2), z.mx4_quantize(normal(o, k, "bf16", 2, 0.02))
    kept = z.MX8(torch.zeros(t, 208, dtype=torch.uint8, device="cuda"), torch.zeros(t, 9, dtype=torch.uint8, device="cuda"), t, k)
    z.mx8_quantize(normal(t, k, "bf16", 3), out=kept)
    flat = torch.full((o * k + 16,), 5, dtype=torch.bfloat16, device="cuda")
    dw = flat[8:8 + o * k].view(o, k)
    dx = torch.empty(t, k, dtype=torch.float16, device="cuda")
    got = z.mx4_linear_backward(dy, kept, w, dx=dx, dw=dw)
    assert got[0] is dx and got[1] is dw
    want = z.mx4_linear_backward(dy, z.mx8_dequantize(kept, torch.float32), w)
    assert torch.equal(dx, want[0].half()) and torch.equal(dw, want[1].bfloat16())
    assert (flat[:8] == 5).all() and (flat[8 + o * k:] == 5).all()


def test_a_checkpoint_with_blocks_that_are_not_numbers(z):
    t, o, k = 70, 64, 64
    x = normal(t, k, "bf16", 3)
    x[5, 3] = float("nan")
    x[66, 40] = float("inf")
    dy, w = normal(t, o, "bf16", 1), z.mx4_quantize(normal(o, k, "bf16", 2))
    kept = z.mx8_quantize(x)
    dx, dw = z.mx4_linear_backward(dy, kept, w)
    want_dx, want_dw = z.mx4_linear_backward(dy, z.mx8_dequantize(kept), w)
    same_values(dx, want_dx, "dx")
    same_values(dw, want_dw, "dw")
    assert torch.isfinite(dx).all() and torch.isnan(dw).any()


def test_no_tokens(z):
    w = z.mx4_quantize(normal(64, 96, "bf16", 2))
    dx, dw = z.mx4_linear_backward(normal(0, 64, "bf16", 1), z.mx8_quantize(normal(0, 96, "bf16", 1)), w)
    assert tuple(dx.shape) == (0, 96) and not dw.any()


def test_wrappers_refuse_what_does_not_fit(z):
    x, w = normal(8, 64, "bf16", 1), z.mx4_quantize(normal(32, 64, "bf16", 2))
    for call in (lambda: z.mx8_quantize(x.t()), lambda: z.mx8_quantize(x.double()), lambda: z.mx8_quantize(x[0]),
                 lambda: z.mx8_quantize(x, out=z.mx8_empty(8, 65)), lambda: z.mx8_quantize(x, out=z.mx4_empty(8, 64)),
                 lambda: z.mx8_dequantize(z.mx8_quantize(x), out=x[:7]),
                 lambda: z.mx4_linear_backward(normal(9, 32, "bf16", 1), z.mx8_quantize(x), w),
                 lambda: z.mx4_linear_backward(normal(8, 32, "bf16", 1), z.mx8_quantize(x[:, :32].contiguous()), w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(z.ZeroError):
        z.mx8_quantize(x[0].expand(8, 64))  # rows on top of one another
