"""GPU tests of the order of MX4 products after the work that writes their
weight, with nothing between the two.  A product of more than 16 tokens is
launched while the tokens are still being quantised and loads the weight before
it waits for them, when the weight's rows of scales lie on 16 bytes: that may
not run ahead of the kernel before those two."""
import pytest
import torch

from test_gpu_mx4 import _normal

pytestmark = pytest.mark.gpu

PASSES = 8


@pytest.fixture(scope="module")
def z():
    import zero_sharded_optimizer_sm_b200 as z

    return z


# 512 columns: rows of scales on 16 bytes; 768: on 8
@pytest.mark.parametrize("tokens", [1, 7, 40, 200])
@pytest.mark.parametrize("o,k", [(2304, 768), (2304, 512), (8192, 2048)])
def test_linear_right_after_the_gather_of_its_weight(z, tokens, o, k):
    n_ranks = 4
    opt = z.ZeroOptimizer([o * k], [0], n_ranks, z.ZERO_STAGE_3, grad_buffers=False)
    opt.view(z.ZERO_VIEW_MASTER).zero_()
    opt.load_master()
    params = opt.view(z.ZERO_VIEW_PARAM)[:o * k].view(torch.bfloat16)
    codes = torch.zeros(n_ranks, o, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n_ranks, o, k // 32, dtype=torch.uint8, device="cuda")
    x = _normal(tokens, k, "bf16", 1)
    news = [_normal(1, o * k, "bf16", 20 + i, 0.02 * 4 ** i)[0] for i in range(PASSES)]
    want = [z.mx4_linear(x, z.mx4_quantize(p.view(o, k))) for p in news]
    torch.cuda.synchronize()
    got = []
    for p in news:
        params.copy_(p)
        opt.all_gather_mx4(0, o * k, codes, scales)
        # the last ranks' first: their buffers are written last
        got.append([z.mx4_linear(x, z.MX4(codes[r], scales[r], o, k)) for r in reversed(range(n_ranks))])
    for ys, y in zip(got, want):
        for a in ys:
            assert torch.equal(a, y)
    opt.close()


@pytest.mark.parametrize("tokens", [1, 7, 40, 200])
@pytest.mark.parametrize("by", ["quantize", "quantize columns", "transpose"])
@pytest.mark.parametrize("o,k", [(2304, 512), (2300, 768), (8192, 2048)])
def test_products_right_after_a_kernel_that_ends_early(z, tokens, by, o, k):
    """The weight written by the quantising kernels, which let the next launch
    start before they end, in the matrix that the last pass's product read;
    forward, backward and the plain product."""
    x, dy = _normal(tokens, k, "bf16", 1), _normal(tokens, o, "bf16", 2)
    xq = z.mx4_quantize(x)
    if by == "quantize":
        sources = [_normal(o, k, "bf16", 20 + i, 0.02 * 4 ** i) for i in range(PASSES)]
        write = lambda s, w: z.mx4_quantize(s, out=w)  # noqa: E731
    elif by == "quantize columns":
        sources = [_normal(k, o, "bf16", 20 + i, 0.02 * 4 ** i) for i in range(PASSES)]
        write = lambda s, w: z.mx4_quantize(s, transpose=True, out=w)  # noqa: E731
    else:
        sources = [z.mx4_quantize(_normal(k, o, "bf16", 20 + i, 0.02 * 4 ** i)) for i in range(PASSES)]
        write = lambda s, w: z.mx4_transpose(s, out=w)  # noqa: E731
    products = [lambda w: z.mx4_linear(x, w), lambda w: z.mx4_linear_backward(dy, x, w)[0], lambda w: z.mx4_matmul(xq, w)]
    for product in products:
        want = []
        for s in sources:
            w = write(s, z.mx4_empty(o, k))
            torch.cuda.synchronize()
            want.append(product(w))
            torch.cuda.synchronize()
        w, got = z.mx4_empty(o, k), []
        for s in sources:
            write(s, w)
            got.append(product(w))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    z.mx4_check()
