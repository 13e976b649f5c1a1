"""mx_linear's out_dtype and out have to agree."""
import pytest
import torch

import mamba_selective_state_amd as ssu


@pytest.mark.parametrize("pair", [False, True])
def test_out_dtype_and_out(pair):
    x = (torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)) if pair else torch.zeros(2, 64)
    w, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    out = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="out_dtype is torch.float32, out has torch.bfloat16"):
        ssu.mx_linear(x, w, s, out=out, out_dtype=torch.float32)
    # that agree: refused for what these tensors are, on the CPU
    with pytest.raises(ValueError, match="GPU"):
        ssu.mx_linear(x, w, s, out=out, out_dtype=torch.bfloat16)
