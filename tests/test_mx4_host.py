"""CPU tests of the MX4 operators' argument checks (zero_mx4_*): every refusal
comes before any device work, with a message, through the C ABI and through
the Python wrappers."""
import ctypes

import pytest
import torch

import mx4_reference as ref
import zero_sharded_optimizer_sm_b200 as z

A = 1 << 20  # stands for a device address; no call below may get as far as using it


def _m(rows=4, cols=64, codes=A, scales=A, code_pitch=None, scale_pitch=None):
    nb = -(-cols // 32)
    return z.zero_mx4(codes, scales, rows, cols, 16 * nb if code_pitch is None else code_pitch,
                      nb if scale_pitch is None else scale_pitch)


def _refused(st, *words):
    assert st == z.ZERO_EINVAL
    msg = z.zero_last_error(None).decode()
    assert msg and all(w in msg for w in words), msg


BAD = [
    (dict(codes=None), "codes"),
    (dict(scales=None), "scales"),
    (dict(codes=A + 8), "16-byte"),
    (dict(code_pitch=24), "code_pitch"),
    (dict(code_pitch=16), "code_pitch"),
    (dict(scale_pitch=1), "scale_pitch"),
    (dict(rows=-1), "out of range"),
    (dict(cols=1 << 31, code_pitch=1 << 40, scale_pitch=1 << 40), "out of range"),
]


@pytest.mark.parametrize("kw,word", BAD)
def test_malformed_matrices_are_refused_everywhere(kw, word):
    bad, n = _m(**kw), ctypes.c_int64()
    good = _m(rows=max(bad.rows, 1), cols=bad.cols if bad.cols < 1 << 30 else 64)
    _refused(z.zero_mx4_dequantize(bad, A, z.ZERO_DTYPE_BF16, 1 << 32, None), word)
    _refused(z.zero_mx4_transpose(bad, z.ZERO_MX4_NEAREST, 0, good, None), "in", word)
    _refused(z.zero_mx4_transpose(good, z.ZERO_MX4_NEAREST, 0, bad, None), "out", word)
    _refused(z.zero_mx4_matmul(bad, good, A, z.ZERO_DTYPE_F32, 1 << 32, A, 1 << 30, None), "a", word)
    _refused(z.zero_mx4_matmul(good, bad, A, z.ZERO_DTYPE_F32, 1 << 32, A, 1 << 30, None), "b", word)
    _refused(z.zero_mx4_matmul_workspace(bad, good, n), word)
    _refused(z.zero_mx4_linear(A, z.ZERO_DTYPE_BF16, 3, 64, bad, A, z.ZERO_DTYPE_BF16, 64, A, 1 << 30, None), "w", word)
    _refused(z.zero_mx4_linear_workspace(3, bad, n), word)
    rows, cols = (bad.rows, bad.cols) if bad.rows >= 0 and bad.cols < 1 << 31 else (4, 64)
    _refused(z.zero_mx4_quantize(A, z.ZERO_DTYPE_BF16, rows, cols, cols, z.ZERO_MX4_NEAREST, 0, bad, None, None), word)
    _refused(z.zero_mx4_quantize(A, z.ZERO_DTYPE_BF16, cols, rows, rows, z.ZERO_MX4_NEAREST, 0, None, bad, None), word)


def test_null_matrices_are_refused():
    n = ctypes.c_int64()
    _refused(z.zero_mx4_dequantize(None, A, 0, 64, None), "in is NULL")
    _refused(z.zero_mx4_transpose(_m(), 0, 0, None, None), "out is NULL")
    _refused(z.zero_mx4_matmul(None, _m(), A, 0, 64, None, 0, None), "a is NULL")
    _refused(z.zero_mx4_linear(A, 0, 3, 64, None, A, 0, 64, A, 1 << 30, None), "w is NULL")
    _refused(z.zero_mx4_quantize(A, 0, 4, 64, 64, 0, 0, None, None, None), "neither")
    _refused(z.zero_mx4_matmul_workspace(_m(), _m(), None), "bytes is NULL")
    _refused(z.zero_mx4_linear_workspace(-1, _m(), n), "-1 tokens")


@pytest.mark.parametrize("kw,word", [
    (dict(src=None), "src"), (dict(src=A + 1), "aligned"), (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"),
    (dict(ld=63), "63"), (dict(rounding=2), "rounding"), (dict(rows=5), "5 x 64"), (dict(cols=65, ld=65), "4 x 65"),
    (dict(rows=-1), "out of range"), (dict(cols=1 << 31, ld=1 << 31), "out of range"),
])
def test_quantize_arguments(kw, word):
    a = dict(src=A, dtype=0, rows=4, cols=64, ld=64, rounding=0)
    a.update(kw)
    _refused(z.zero_mx4_quantize(a["src"], a["dtype"], a["rows"], a["cols"], a["ld"], a["rounding"], 0, _m(), None, None), word)


def test_shapes_that_do_not_fit():
    _refused(z.zero_mx4_quantize(A, 0, 4, 64, 64, 0, 0, None, _m(), None), "out_t is not 64 x 4")
    _refused(z.zero_mx4_transpose(_m(), 0, 0, _m(), None), "out is not 64 x 4")
    _refused(z.zero_mx4_transpose(_m(), 7, 0, _m(rows=64, cols=4), None), "rounding")
    _refused(z.zero_mx4_matmul(_m(), _m(cols=96), A, 0, 64, None, 0, None), "64 columns, b 96")
    _refused(z.zero_mx4_matmul(_m(), _m(rows=9), A, 0, 8, None, 0, None), "out: 8 elements")
    _refused(z.zero_mx4_matmul(_m(), _m(), A + 1, 0, 64, None, 0, None), "out is null or not aligned")
    _refused(z.zero_mx4_matmul(_m(), _m(), A + 2, z.ZERO_DTYPE_F32, 64, None, 0, None), "out is null or not aligned")
    _refused(z.zero_mx4_matmul(_m(), _m(), A, 5, 64, None, 0, None), "dtype")
    _refused(z.zero_mx4_linear(A, 0, 3, 60, _m(), A, 0, 64, A, 1 << 30, None), "x: 60")
    _refused(z.zero_mx4_linear(A, 0, 3, 64, _m(), A, 0, 3, A, 1 << 30, None), "y: 3")
    _refused(z.zero_mx4_linear(A, 0, -2, 64, _m(), A, 0, 64, A, 1 << 30, None), "out of range")


@pytest.mark.parametrize("kw,word", [
    (dict(dy=None), "dy"), (dict(x=None), "x is null"), (dict(dx=None), "dx"), (dict(dw=None), "dw"),
    (dict(dy_dtype=3), "dtype"), (dict(x_dtype=-1), "dtype"), (dict(dx_dtype=9), "dtype"), (dict(dw_dtype=9), "dtype"),
    (dict(ld_dy=3), "dy: 3"), (dict(ld_x=63), "x: 63"), (dict(ld_dx=63), "dx: 63"), (dict(ld_dw=63), "dw: 63"),
    (dict(rounding=5), "rounding"), (dict(tokens=-1), "out of range"), (dict(workspace=None), "workspace"),
    (dict(workspace=A + 4), "workspace"), (dict(bytes=100), "workspace"), (dict(w=None), "w is NULL"),
    (dict(w=_m(code_pitch=8)), "w: code_pitch"),
])
def test_linear_backward_arguments(kw, word):
    a = dict(dy=A, dy_dtype=0, ld_dy=4, x=A, x_dtype=0, ld_x=64, tokens=5, w=_m(), rounding=0, seed=0, dx=A, dx_dtype=0,
             ld_dx=64, dw=A, dw_dtype=0, ld_dw=64, workspace=A, bytes=1 << 20)
    a.update(kw)
    _refused(z.zero_mx4_linear_backward(*a.values(), None), word)


def test_linear_backward_workspace():
    """dy (5 x 4), its transpose, x's (64 x 5) and w's (64 x 4): one block of
    codes and 16 bytes of scales to a row of each."""
    n = ctypes.c_int64()
    assert z.zero_mx4_linear_backward_workspace(5, _m(), n) == 0 and n.value == 32 * (5 + 4 + 64 + 64)
    assert z.zero_mx4_linear_backward_workspace(0, _m(), n) == 0 and n.value == 0
    _refused(z.zero_mx4_linear_backward_workspace(-1, _m(), n), "tokens")
    _refused(z.zero_mx4_linear_backward_workspace(5, _m(), None), "NULL")


def test_empty_matrices_do_nothing():
    e = _m(rows=0, codes=None, scales=None)
    n = ctypes.c_int64(-1)
    assert z.zero_mx4_quantize(None, 0, 0, 64, 64, 0, 0, e, None, None) == 0
    assert z.zero_mx4_dequantize(e, None, 0, 64, None) == 0
    assert z.zero_mx4_transpose(e, 0, 0, _m(rows=64, cols=0, codes=None, scales=None), None) == 0
    assert z.zero_mx4_matmul(e, _m(), None, 0, 4, None, 0, None) == 0
    assert z.zero_mx4_linear(None, 0, 0, 64, _m(), None, 0, 4, None, 0, None) == 0
    assert z.zero_mx4_linear_workspace(0, _m(), n) == 0 and n.value == 0


@pytest.mark.parametrize("rows,cols,pitch,want", [
    (1, 32, 16, 0), (300, 512, 16, 0), (300, 512, 32, 0),   # rows of scales on 16 bytes: loaded as they lie
    (300, 512, 17, 4 * 2048), (1, 513, 17, 2 * 2 * 2048), (257, 1024, 33, 4 * 2 * 2048),
])
def test_workspace_of_a_matrix(rows, cols, pitch, want):
    """2048 bytes for each 128 rows (in whole pairs) and 512 columns of a
    matrix whose rows of scales are not 16-byte aligned."""
    n = ctypes.c_int64()
    m, other = _m(rows, cols, scale_pitch=pitch), _m(8, cols, scale_pitch=64)
    assert z.zero_mx4_matmul_workspace(m, other, n) == 0 and n.value == want
    assert z.zero_mx4_matmul_workspace(other, m, n) == 0 and n.value == want
    nb = ref.blocks_of(cols)
    assert z.zero_mx4_linear_workspace(40, m, n) == 0
    assert n.value == want + 40 * (16 * nb + (nb + 15) // 16 * 16)
    assert z.zero_mx4_linear_workspace(16, m, n) == 0  # x is quantised inside the product
    assert n.value == (want if pitch % 4 else 0)


def test_a_short_workspace_is_refused():
    """Before any launch: the call needs the device's properties first, so
    without a device it stops there instead."""
    m = _m(scale_pitch=3)
    st = z.zero_mx4_matmul(m, m, A, 0, 64, None, 0, None)
    assert st == (z.ZERO_EINVAL if torch.cuda.is_available() else z.ZERO_ECUDA)


def test_collectives_need_a_bound_context():
    lay = z.zero_layout(1, (ctypes.c_int64 * 1)(64), (ctypes.c_int32 * 1)(0))
    ctx = ctypes.c_void_p()
    assert z.zero_init(ctypes.byref(lay), 2, 2, 0, ctypes.byref(ctx)) == 0
    try:
        ptrs = (ctypes.c_void_p * 2)(A, A)
        for fn in (z.zero_mx4_all_gather, z.zero_mx4_reduce_scatter):
            assert fn(ctx, 0, 64, ptrs, ptrs, None) == z.ZERO_ESTATE
            assert "not bound" in z.zero_last_error(ctx).decode()
            assert fn(None, 0, 64, ptrs, ptrs, None) == z.ZERO_EINVAL
    finally:
        z.zero_destroy(ctx)


def test_option_dtype_refuses_binary32():
    lay = z.zero_layout(1, (ctypes.c_int64 * 1)(64), (ctypes.c_int32 * 1)(0))
    ctx = ctypes.c_void_p()
    assert z.zero_init(ctypes.byref(lay), 2, 2, 0, ctypes.byref(ctx)) == 0
    try:
        assert z.zero_set_option(ctx, z.ZERO_OPT_DTYPE, z.ZERO_DTYPE_F32) == z.ZERO_EINVAL
    finally:
        z.zero_destroy(ctx)


# ---------------------------------------------------------- the wrappers --

def test_wrappers_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64)
    for call in (lambda: z.mx4_quantize(x), lambda: z.mx4_quantize_both(x), lambda: z.mx4_quantize(x, transpose=True)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        z.MX4(codes, scales, 4, 64)
    with pytest.raises(ValueError, match="codes"):
        z.MX4(codes.float(), scales, 4, 64)
    with pytest.raises(ValueError, match="codes"):
        z.MX4(codes[:, :16], scales, 4, 64)
    with pytest.raises(ValueError, match="scales"):
        z.MX4(codes, scales[:, :1], 4, 64)
    with pytest.raises(ValueError, match="codes"):
        z.MX4(codes[:3], scales, 4, 64)
    with pytest.raises(ValueError, match="contiguous"):
        z.MX4(torch.zeros(4, 64, dtype=torch.uint8)[:, ::2], scales, 4, 64)
    with pytest.raises(ValueError):
        z.mx4_empty(-1, 64)


# ------------------------------------------------- the reference itself --

def test_reference_rounds_to_the_nearest_grid_value():
    """Against a search over the grid, ties to the even code."""
    x = torch.linspace(-8, 8, 32 * 41, dtype=torch.float64).view(41, 32)
    x = torch.cat([x, x * 2.0 ** -20, x * 1000, torch.zeros(1, 32, dtype=torch.float64)])
    code, s = ref.quantize(x)
    for row in range(x.shape[0]):
        m = x[row].abs().max()
        want_s = 0 if m == 0 else max(int(torch.frexp(m)[1]) - 1 - 2 + 127, 0)
        assert int(s[row, 0]) == want_s
        for j in range(32):
            a = abs(float(x[row, j])) / 2.0 ** (want_s - 127)
            best = min(range(8), key=lambda c: (abs(ref.MAGNITUDES[c] - a), c % 2))
            assert int(code[row, 0, j]) % 8 == best


def test_reference_random_numbers_are_philox():
    """The generator's published known answer: counter 0, key 0."""
    r = ref.random16(1, 0)[0, :8].tolist()
    words = [r[2 * i] | r[2 * i + 1] << 16 for i in range(4)]
    assert words == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
