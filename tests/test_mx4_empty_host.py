"""CPU tests of where MX4 matrices may lie."""
import pytest
import torch

import zero_sharded_optimizer_sm_b200 as z


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"])
@pytest.mark.parametrize("rows", [0, 4])
def test_an_mx4_matrix_is_not_made_off_the_gpu(device, rows):
    """A kernel would be handed its addresses."""
    with pytest.raises(ValueError, match="CUDA"):
        z.mx4_empty(rows, 64, device=device)
