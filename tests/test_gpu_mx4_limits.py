"""GPU test of an MX4 matrix of as many rows as there may be."""
import pytest
import torch

import mx4_reference as ref
from test_gpu_mx4 import _assert_mx4, _same_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1])
def test_the_greatest_number_of_rows(cols):
    """2^31 - 256 rows (each one block): quantised and read back at both ends
    and in between."""
    import zero_sharded_optimizer_sm_b200 as z

    rows = 2 ** 31 - 256
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = [0, 2 ** 30 - 20, 2 ** 31 - 2 ** 24 - 20, rows - 40]
    g = torch.Generator("cuda").manual_seed(1)
    for i in at:
        x[i:i + 40] = torch.randn(40, cols, generator=g, device="cuda")
    out = z.MX4(torch.empty(rows, 16, dtype=torch.uint8, device="cuda"),
                torch.empty(rows, 1, dtype=torch.uint8, device="cuda"), rows, cols)
    z.mx4_quantize(x, out=out)
    for i in at:
        part = z.MX4(out.codes[i:i + 40], out.scales[i:i + 40], 40, cols)
        _assert_mx4(part, *ref.quantize(x[i:i + 40]), f"row {i}")
    back = z.mx4_dequantize(out)
    for i in at:
        _same_values(back[i:i + 40], ref.rounded(x[i:i + 40]), f"row {i} read back")
    assert (back[at[0] + 40:at[0] + 4096] == 0).all() and (out.codes[at[1] + 40:at[1] + 4096] == 0).all()
