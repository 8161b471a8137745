"""GPU tests of calls around a layer's products at the edges of their ranges:
rows without columns, tables without rows."""
import pytest
import torch

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
