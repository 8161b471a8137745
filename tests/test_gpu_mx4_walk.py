"""GPU tests of the MX4 products whose CTAs walk several tiles one after
another without CTA pairs: few tokens through a weight of a vocabulary's size
(2 to 16 tokens over more than 2 * 148 * 128 outputs, 17 to 128 over more than
148 * 128)."""
import pytest
import torch

import mx4_reference as ref
from test_gpu_mx4 import DTYPES, _assert_product, _normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


def _weights(z, out, inner):
    """The same weight with rows of scales on 16 bytes and end to end."""
    w = z.mx4_quantize(_normal(out, inner, "bf16", out + inner, 0.02))
    return w, z.MX4(w.codes, w.scales[:, :ref.blocks_of(inner)].contiguous(), out, inner)


# k tiles of 256: 3, 1, 5, 4, 7
@pytest.mark.parametrize("out,inner", [(50304, 768), (50304, 200), (40001, 1100), (38000, 896), (80000, 1600)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_few_tokens_through_many_outputs(z, dtype, out, inner):
    """Against 64-bit arithmetic and, bit for bit, against the product of the
    quantised tokens, which the kernel does not quantise itself; every run the
    same.  Scale rows that load as they lie, by words and as pieces."""
    weights = _weights(z, out, inner)
    for tokens in (2, 7, 16):
        x = _normal(tokens, inner, dtype, tokens)
        # each token and each block of its own size, so that scales of another k tile or row would show
        x *= 2.0 ** torch.randint(-6, 7, (tokens, 1), device="cuda", generator=torch.Generator("cuda").manual_seed(tokens))
        x *= 2.0 ** (torch.arange(inner, device="cuda") // 32 % 9 - 4)
        xq = z.mx4_quantize(x)
        want = z.mx4_matmul(xq, weights[0], x.dtype)
        _assert_product(want, xq, weights[0], "product")
        for w in weights:
            for _ in range(10):
                assert torch.equal(z.mx4_linear(x, w), want)
    z.mx4_check()


@pytest.mark.parametrize("tokens,out,inner", [(17, 20000, 768), (40, 20001, 200), (100, 50304, 768), (128, 19000, 1100),
                                              (64, 38001, 520)])
def test_a_small_batch_through_many_outputs(z, tokens, out, inner):
    x = _normal(tokens, inner, "bf16", 3)
    xq = z.mx4_quantize(x)
    for w in _weights(z, out, inner):
        got = z.mx4_linear(x, w)
        _assert_product(got, xq, w, "linear")
        for _ in range(5):
            assert torch.equal(z.mx4_linear(x, w), got)
        assert torch.equal(z.mx4_matmul(xq, w), got)
    z.mx4_check()
