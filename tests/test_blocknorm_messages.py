"""CPU test: a refusal of the block norm's gradients names the operand that it is about."""
import pytest
import torch

import thread_register_tile_amd as trt


@pytest.mark.parametrize("name", ["dh", "dr_out"])
def test_upstream_gradient_is_named(name):
    up, y = torch.zeros(70, 4).t(), torch.zeros(4, 70)
    with pytest.raises(trt.TrtError, match=f"{name} must have unit inner stride") as e:
        trt.block_norm_bwd(up if name == "dh" else None, up if name == "dr_out" else None, y, y)
    assert e.value.status == trt.ERR_STRIDE
