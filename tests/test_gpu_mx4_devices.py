"""GPU tests of the MX4 collectives of a context whose device was named in any
of torch's ways."""
import pytest
import torch

import mx4_reference as ref
from test_gpu_mx4 import _assert_mx4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("device", [None, "cuda", "cuda:0", torch.device("cuda"), 0])
@pytest.mark.parametrize("own_stream", [False, True])
def test_collectives_of_a_context_on_a_named_device(device, own_stream):
    import zero_sharded_optimizer_sm_b200 as z

    n, ranks = 4096, 2
    opt = z.ZeroOptimizer([n], [0], ranks, z.ZERO_STAGE_2, grad_buffers=False, device=device)
    opt.view(z.ZERO_VIEW_MASTER).copy_(torch.randn(n, device="cuda"))
    opt.load_master()
    codes = torch.zeros(ranks, n // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(ranks, n // 32, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    kw = dict(stream=torch.cuda.Stream()) if own_stream else {}
    opt.all_gather_mx4(0, n, codes, scales, **kw)
    torch.cuda.synchronize()
    want = opt.view(z.ZERO_VIEW_MASTER).to(torch.bfloat16).view(1, n)
    for r in range(ranks):
        _assert_mx4(z.MX4(codes[r].view(1, -1), scales[r].view(1, -1), 1, n), *ref.quantize(want), f"rank {r}")
    opt.reduce_scatter_mx4(0, n, codes, scales, **kw)
    torch.cuda.synchronize()
    shard = opt.view(z.ZERO_VIEW_GRAD_SHARD)[:n].view(torch.bfloat16)
    assert torch.equal(shard.double(), ref.rounded(want)[0])  # the mean of two equal gradients
    opt.close()
