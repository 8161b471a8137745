"""GPU tests of calls around a layer's products at the edges of their ranges:
rows without columns, tables without rows, results whose rows are far apart."""
import pytest
import torch

from test_gpu_mx8 import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def test_rstd_of_rows_without_columns(z):
    """The mean of nothing is not a number; the result is written all the same."""
    x, w = torch.empty(300, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(), dict(residual=x), dict(rstd=torch.full((300,), 5.0, device="cuda")), dict(y8=True)):
        n = z.rms_norm(x, w, **kw)
        assert tuple(n.rstd.shape) == (300,) and torch.isnan(n.rstd).all()
        assert tuple(n.y.shape) == (300, 0)
    beside = torch.full((10,), 5.0, device="cuda")
    z.rms_norm(x[:4], w, rstd=beside[3:7])
    assert torch.isnan(beside[3:7]).all() and (beside[:3] == 5).all() and (beside[7:] == 5).all()


@pytest.mark.parametrize("dtype", [0, 2, -1, 99])
def test_an_mx4_table_without_rows(z, dtype):
    """Every token is padding; the dense table's type is not looked at."""
    t = torch.tensor([0, 5, -1], device="cuda")
    big = torch.full((3, 70), 7.0, dtype=torch.float16, device="cuda")
    for codes in (None, big.data_ptr()):
        big.fill_(7)
        empty = z.zero_mx4(codes, codes, 0, 64, 32, 2)
        st = z.zero_embedding(t.data_ptr(), 8, 3, None, dtype, 0, 64, 0, empty, 1.0, big.data_ptr(), z.ZERO_DTYPE_F16, 70,
                              torch.cuda.current_stream().cuda_stream)
        assert st == 0, z.zero_last_error(None).decode()
        assert not big[:, :64].any() and (big[:, 64:] == 7).all()
    m = z.MX4(torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda"), 0, 64)
    assert not z.embedding(t, m).any()


def test_zeros_into_rows_that_are_far_apart(z):
    """A gradient of no tokens, whose rows are more than 2^31 bytes apart; and one
    row of more."""
    pitch = (1 << 30) + 72
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("wants 8 GB")
    memory = torch.full((2 * pitch,), 3.0, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    table = memory.as_strided((2, 40), (pitch, 1))
    z.embedding_backward(normal(0, 40, "bf16", 1), none, 2, out=table)
    assert not table.any() and (memory[40:80] == 3).all() and (memory[pitch + 40:pitch + 80] == 3).all()
    table.fill_(3)
    w = z.mx4_quantize(normal(2, 40, "bf16", 2))
    z.mx4_linear_backward(normal(0, 2, "bf16", 1), normal(0, 40, "bf16", 1), w, dw=table)
    assert not table.any() and (memory[40:80] == 3).all()
    wide = memory[:(1 << 30) + 9]
    x = torch.empty(0, wide.shape[0], dtype=torch.bfloat16, device="cuda")
    z.rms_norm_backward(x, x, wide, none.float(), dw=wide)
    assert not wide.any() and memory[(1 << 30) + 9] == 3
