"""GPU tests of the order in which the table gradient adds a token's rows: the
same whether the call writes the table or adds to it."""
import pytest
import torch

from test_gpu_embedding import tokens_of
from test_gpu_mx8 import DTYPES, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [8, 260, 771])
@pytest.mark.parametrize("n", [40, 100, 300, 511, 512, 513, 5000])
def test_adding_to_zeros_is_writing(z, n, cols, dtype):
    """Numbers whose sum depends on the order, one token at most places."""
    dy, vocab = normal(n, cols, "f32", n).to(DTYPES[dtype]), 50
    dy[::3] *= 1000
    t = tokens_of(n, vocab, 3, "outside")
    t[2:n - 3] = torch.where(t[2:n - 3] % 4 == 0, t[2:n - 3], 7)
    written = z.embedding_backward(dy, t, vocab, 1.5, out=torch.empty(vocab, cols, device="cuda"))
    added = z.embedding_backward(dy, t, vocab, 1.5, out=torch.zeros(vocab, cols, device="cuda"), accumulate=True)
    assert torch.equal(added, written)


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z
