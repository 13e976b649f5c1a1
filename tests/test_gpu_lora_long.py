"""add_lora over rows so long that a byte's place in them passes 32 bits: one row under many numbers (stride 0), so that
a few GB hold it. x and A are 0 but at five places, where they are powers of two; so h is exact."""
import pytest
import torch

import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,k", [(torch.float32, 720_000_064), (torch.bfloat16, 1_440_000_128)])
@pytest.mark.parametrize("rows", [3, 257])
def test_long_rows(dt, k, rows):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    print("[gpu] add_lora", rows, "rows of", k, dt, flush=True)
    x, a = torch.zeros(k, dtype=dt, device="cuda"), torch.zeros(1, 1, k, dtype=dt, device="cuda")
    at = torch.tensor([0, k // 4 + 1, k // 2, 3 * (k // 4), k - 1], device="cuda")
    x[at] = 2.0 ** torch.arange(5, device="cuda").to(dt)
    a[0, 0, at] = 1
    b = torch.tensor([1.0, -2.0, 0.5], dtype=dt, device="cuda").view(1, 3, 1)
    y = torch.zeros(rows, 3, dtype=dt, device="cuda")
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ids[1] = -1
    ssu.add_lora(y, x.expand(rows, k), a, b, ids)
    want = torch.tensor([31.0, -62.0, 15.5], dtype=dt, device="cuda").repeat(rows, 1)
    want[1] = 0
    assert torch.equal(y, want)
