"""The layer operators on a GPU that is not the current one: they run there, in the order of that
GPU's current stream, and leave the current GPU as it was."""
import pytest
import torch

import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpus():
    if not torch.cuda.is_available() or torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")


def calls(dev):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(40, 512, generator=g).bfloat16().to(dev)
    w = torch.randn(96, 512, generator=g).to(dev)
    logits = (3 * torch.randn(2, 60000, generator=g)).to(dev)
    codes = ssu.mx_quantize(w)
    y, u = ssu.add_rms_norm(x, torch.ones(512, dtype=torch.bfloat16, device=dev), residual=x)
    r = ssu.token_logprobs(logits, torch.tensor([5, 7], device=dev), 4)
    return [*codes, y, u, ssu.mx_linear(x, *codes), *r]


@pytest.mark.parametrize("own_stream", [False, True])
def test_second_gpu(own_stream):
    with torch.cuda.device(0):
        want = calls("cuda:0")
        torch.cuda.synchronize(0)
        if own_stream:
            with torch.cuda.device(1):
                s = torch.cuda.Stream()
                torch.cuda.set_stream(s)
        got = calls("cuda:1")
        assert torch.cuda.current_device() == 0
        torch.cuda.synchronize(1)
    for a, b in zip(got, want):
        assert a.device.index == 1 and torch.equal(a.cpu(), b.cpu())
    if own_stream:
        with torch.cuda.device(1):
            torch.cuda.set_stream(torch.cuda.default_stream())
