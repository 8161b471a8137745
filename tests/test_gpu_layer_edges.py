"""GPU tests of calls around a layer's products at the edges of their ranges:
rows without columns."""
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
