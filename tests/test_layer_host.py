"""CPU tests of the argument checks of the calls around a layer's products
(zero_mx8_*, zero_rms_norm*, zero_embedding*): every refusal comes before any
device work, with a message, through the C ABI and through the Python wrappers."""
import ctypes

import pytest
import torch

import zero_sharded_optimizer_sm_b200 as z

A = 1 << 20  # stands for a device address; no call below may get as far as using it
BF16, F16, F32 = z.ZERO_DTYPE_BF16, z.ZERO_DTYPE_F16, z.ZERO_DTYPE_F32


def _m8(rows=4, cols=64, codes=A, scales=A, code_pitch=None, scale_pitch=None):
    nb = -(-cols // 32)
    return z.zero_mx8(codes, scales, rows, cols, 32 * nb if code_pitch is None else code_pitch,
                      nb if scale_pitch is None else scale_pitch)


def _m4(rows=4, cols=64):
    nb = -(-cols // 32)
    return z.zero_mx4(A, A, rows, cols, 16 * nb, nb)


def _refused(st, *words):
    assert st == z.ZERO_EINVAL
    msg = z.zero_last_error(None).decode()
    assert msg and all(w in msg for w in words), msg


BAD = [
    (dict(codes=None), "codes"), (dict(scales=None), "scales"), (dict(codes=A + 8), "16-byte"),
    (dict(code_pitch=72), "code_pitch"), (dict(code_pitch=48), "code_pitch"), (dict(scale_pitch=1), "scale_pitch"),
    (dict(rows=-1), "out of range"), (dict(cols=1 << 31, code_pitch=1 << 40, scale_pitch=1 << 40), "out of range"),
]


def norm_args(**kw):
    a = dict(x=A, residual=None, dtype=BF16, rows=4, cols=64, ld_x=64, ld_residual=64, weight=A, weight_dtype=BF16, eps=1e-6,
             y=A, ld_y=64, h=None, ld_h=64, y8=None, h8=None, rstd=None)
    a.update(kw)
    return list(a.values()) + [None]


def back_args(**kw):
    a = dict(dy=A, dtype=BF16, rows=4, cols=64, ld_dy=64, h=A, ld_h=64, h8=None, weight=A, weight_dtype=BF16, rstd=A, dh=None,
             ld_dh=64, dx=A, ld_dx=64, dw=A, dw_dtype=BF16, workspace=A, bytes=1 << 20)
    a.update(kw)
    return list(a.values()) + [None]


def embed_args(**kw):
    a = dict(tokens=A, token_bytes=8, n=5, table=A, dtype=BF16, vocab=10, cols=64, ld=64, table4=None, scale=1.0, out=A,
             out_dtype=BF16, ld_out=64)
    a.update(kw)
    return list(a.values()) + [None]


def embed_back_args(**kw):
    a = dict(dy=A, dtype=BF16, n=5, cols=64, ld_dy=64, tokens=A, token_bytes=8, vocab=10, scale=1.0, dtable=A,
             dtable_dtype=BF16, ld=64, accumulate=0, workspace=A, bytes=1 << 20)
    a.update(kw)
    return list(a.values()) + [None]


def saved_args(**kw):
    a = dict(dy=A, dy_dtype=BF16, ld_dy=4, x=_m8(rows=5), w=_m4(), rounding=0, seed=0, dx=A, dx_dtype=BF16, ld_dx=64, dw=A,
             dw_dtype=BF16, ld_dw=64, workspace=A, bytes=1 << 20)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw,word", BAD)
def test_malformed_matrices_are_refused_everywhere(kw, word):
    bad = _m8(**kw)
    rows, cols = (bad.rows, bad.cols) if bad.rows >= 0 and bad.cols < 1 << 31 else (4, 64)
    _refused(z.zero_mx8_quantize(A, BF16, rows, cols, cols, bad, None), "out", word)
    _refused(z.zero_mx8_dequantize(bad, A, BF16, 1 << 32, None), "in", word)
    _refused(z.zero_rms_norm(*norm_args(y8=bad)), "y8", word)
    _refused(z.zero_rms_norm(*norm_args(h8=bad)), "h8", word)
    _refused(z.zero_rms_norm_backward(*back_args(h=None, h8=bad)), "h8", word)
    _refused(z.zero_mx4_linear_backward_mx8(*saved_args(x=bad)), "x", word)


@pytest.mark.parametrize("kw,word", [
    (dict(src=None), "src"), (dict(src=A + 1), "aligned"), (dict(dtype=3), "dtype"), (dict(ld=63), "63"),
    (dict(rows=5), "5 x 64"), (dict(cols=65, ld=65), "4 x 65"), (dict(rows=-1), "out of range"), (dict(out=None), "NULL"),
])
def test_quantize_arguments(kw, word):
    a = dict(src=A, dtype=0, rows=4, cols=64, ld=64, out=_m8())
    a.update(kw)
    _refused(z.zero_mx8_quantize(*a.values(), None), word)


def test_dequantize_arguments():
    _refused(z.zero_mx8_dequantize(None, A, 0, 64, None), "in is NULL")
    _refused(z.zero_mx8_dequantize(_m8(), None, 0, 64, None), "dst")
    _refused(z.zero_mx8_dequantize(_m8(), A + 2, F32, 64, None), "dst")
    _refused(z.zero_mx8_dequantize(_m8(), A, 7, 64, None), "dtype")
    _refused(z.zero_mx8_dequantize(_m8(), A, 0, 60, None), "60")


@pytest.mark.parametrize("kw,words", [
    (dict(x=None), ["x is null"]), (dict(x=A + 1), ["x", "aligned"]), (dict(dtype=3), ["dtype"]), (dict(ld_x=63), ["x: 63"]),
    (dict(rows=-1), ["out of range"]), (dict(cols=1 << 31, ld_x=1 << 31), ["out of range"]),
    (dict(residual=A + 1), ["residual"]), (dict(residual=A, ld_residual=3), ["residual: 3"]),
    (dict(weight=None), ["weight"]), (dict(weight=A + 2, weight_dtype=F32), ["weight"]), (dict(weight_dtype=-1), ["dtype"]),
    (dict(eps=0.0), ["eps"]), (dict(eps=-1e-6), ["eps"]), (dict(eps=float("nan")), ["eps"]), (dict(eps=float("inf")), ["eps"]),
    (dict(eps=1e-60), ["eps"]), (dict(eps=1e60), ["eps"]),
    (dict(y=None), ["no result"]), (dict(y=A + 1), ["y is null or not"]), (dict(ld_y=60), ["y: 60"]),
    (dict(h=A + 1), ["h is"]), (dict(h=A, ld_h=60), ["h: 60"]), (dict(rstd=A + 2), ["rstd"]),
    (dict(y8=_m8(rows=3)), ["y8 is not 4 x 64"]), (dict(h8=_m8(cols=65)), ["h8 is not 4 x 64"]),
])
def test_norm_arguments(kw, words):
    _refused(z.zero_rms_norm(*norm_args(**kw)), *words)


@pytest.mark.parametrize("kw,words", [
    (dict(dy=None), ["dy"]), (dict(dtype=4), ["dtype"]), (dict(ld_dy=1), ["dy: 1"]), (dict(rows=-2), ["out of range"]),
    (dict(h=None), ["h is null"]), (dict(h8=_m8()), ["both h and h8"]), (dict(ld_h=63), ["h: 63"]),
    (dict(h=None, h8=_m8(rows=9)), ["h8 is not 4 x 64"]), (dict(weight=None), ["weight"]), (dict(weight_dtype=9), ["dtype"]),
    (dict(rstd=None), ["rstd"]), (dict(rstd=A + 2), ["rstd"]), (dict(dh=A + 1), ["dh"]), (dict(dh=A, ld_dh=63), ["dh: 63"]),
    (dict(dx=None), ["dx"]), (dict(ld_dx=63), ["dx: 63"]), (dict(dw=None), ["dw"]), (dict(dw_dtype=5), ["dtype"]),
    (dict(workspace=None), ["workspace"]), (dict(workspace=A + 4), ["workspace"]), (dict(bytes=16), ["workspace"]),
])
def test_norm_backward_arguments(kw, words):
    _refused(z.zero_rms_norm_backward(*back_args(**kw)), *words)


TOKENS = [(dict(tokens=None), ["tokens"]), (dict(tokens=A + 4), ["tokens"]), (dict(token_bytes=2), ["2 bytes"]),
          (dict(n=-1), ["-1 tokens"]), (dict(n=1 << 31), ["tokens"]), (dict(vocab=-1), ["vocabulary"]),
          (dict(vocab=1 << 31), ["vocabulary"]), (dict(scale=float("nan")), ["scale"]), (dict(scale=1e39), ["scale"])]


@pytest.mark.parametrize("kw,words", TOKENS + [
    (dict(table=None), ["table"]), (dict(table=A + 1), ["table"]), (dict(dtype=3), ["dtype"]), (dict(ld=8), ["table: 8"]),
    (dict(table4=_m4(rows=10)), ["both table"]), (dict(table=None, table4=_m4(rows=9)), ["table4 is not 10 x 64"]),
    (dict(out=None), ["out"]), (dict(out_dtype=3), ["dtype"]), (dict(ld_out=63), ["out: 63"]),
    (dict(cols=-1), ["out of range"]), (dict(vocab=0, table=None, out=None), ["out"]),
])
def test_embedding_arguments(kw, words):
    _refused(z.zero_embedding(*embed_args(**kw)), *words)


@pytest.mark.parametrize("kw,words", TOKENS + [
    (dict(dy=None), ["dy"]), (dict(dtype=3), ["dtype"]), (dict(ld_dy=8), ["dy: 8"]), (dict(dtable=None), ["dtable"]),
    (dict(dtable_dtype=3), ["dtype"]), (dict(ld=8), ["dtable: 8"]), (dict(accumulate=2), ["accumulate"]),
    (dict(workspace=None, n=1000), ["workspace"]), (dict(workspace=A + 8, n=1000), ["workspace"]),
    (dict(bytes=8, n=1000), ["workspace"]),
])
def test_embedding_backward_arguments(kw, words):
    _refused(z.zero_embedding_backward(*embed_back_args(**kw)), *words)


@pytest.mark.parametrize("kw,words", [
    (dict(dy=None), ["dy"]), (dict(x=None), ["x is NULL"]), (dict(x=_m8(rows=5, cols=96)), ["x has 96 inputs, w 64"]),
    (dict(w=None), ["w is NULL"]), (dict(dx=None), ["dx"]), (dict(dw=None), ["dw"]), (dict(dy_dtype=3), ["dtype"]),
    (dict(dx_dtype=9), ["dtype"]), (dict(dw_dtype=9), ["dtype"]), (dict(ld_dy=3), ["dy: 3"]), (dict(ld_dx=63), ["dx: 63"]),
    (dict(ld_dw=63), ["dw: 63"]), (dict(rounding=5), ["rounding"]), (dict(workspace=None), ["workspace"]),
    (dict(bytes=100), ["workspace"]),
])
def test_linear_backward_from_a_checkpoint_arguments(kw, words):
    _refused(z.zero_mx4_linear_backward_mx8(*saved_args(**kw)), *words)


def test_workspaces():
    n = ctypes.c_int64(-1)
    assert z.zero_rms_norm_backward_workspace(0, 64, n) == 0 and n.value == 0
    assert z.zero_rms_norm_backward_workspace(3, 64, n) == 0 and n.value > 0
    assert z.zero_embedding_backward_workspace(0, 10, 64, n) == 0 and n.value == 0
    assert z.zero_embedding_backward_workspace(5, 10, 64, n) == 0 and n.value == 0  # (few tokens are not sorted)
    assert z.zero_embedding_backward_workspace(1000, 10, 64, n) == 0 and n.value > 0
    _refused(z.zero_rms_norm_backward_workspace(-1, 64, n), "out of range")
    _refused(z.zero_rms_norm_backward_workspace(3, 64, None), "NULL")
    _refused(z.zero_embedding_backward_workspace(5, 1 << 31, 64, n), "out of range")
    _refused(z.zero_embedding_backward_workspace(5, 10, 64, None), "NULL")


def test_empty_matrices_do_nothing():
    e = _m8(rows=0, codes=None, scales=None)
    assert z.zero_mx8_quantize(None, 0, 0, 64, 64, e, None) == 0
    assert z.zero_mx8_dequantize(e, None, 0, 64, None) == 0
    assert z.zero_rms_norm(*norm_args(rows=0, x=None, y=A)) == 0
    assert z.zero_rms_norm(*norm_args(cols=0, x=None, weight=None)) == 0
    assert z.zero_rms_norm_backward(*back_args(cols=0, dy=None, h=None, weight=None, rstd=None, dx=None, dw=None)) == 0
    assert z.zero_embedding(*embed_args(n=0, tokens=None, out=None)) == 0
    assert z.zero_embedding(*embed_args(cols=0, out=None)) == 0
    assert z.zero_embedding_backward(*embed_back_args(vocab=0, dtable=None)) == 0
    assert z.zero_embedding_backward(*embed_back_args(n=0, tokens=None, dy=None, accumulate=1)) == 0


def test_wrappers_refuse_what_is_not_on_a_gpu():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: z.mx8_quantize(x), lambda: z.rms_norm(x, w), lambda: z.rms_norm_backward(x, x, w, w),
                 lambda: z.embedding(torch.zeros(3, dtype=torch.int64), x),
                 lambda: z.embedding_backward(x, torch.zeros(4, dtype=torch.int64), 9),
                 lambda: z.mx8_empty(4, 64, device="cpu"), lambda: z.MX8(torch.zeros(4, 64, dtype=torch.uint8),
                                                                        torch.zeros(4, 2, dtype=torch.uint8), 4, 64)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("codes,scales,rows,cols", [
    ((4, 63), (4, 2), 4, 64), ((4, 64), (4, 1), 4, 64), ((3, 64), (4, 2), 4, 64), ((4, 64), (4, 2), 4, 65)])
def test_an_mx8_matrix_of_the_wrong_size_is_refused(codes, scales, rows, cols):
    with pytest.raises(ValueError):
        z.MX8(torch.zeros(codes, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8), rows, cols)
