"""beam_select, reorder_states and add_lora together with the state update and the layer operators, as a
search calls them (examples/beam_search.py)."""
import importlib.util
import os

import pytest
import torch

import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_against_plain_torch(example):
    """A step's log probability is off by less than 0.3, as in the decode step (bf16 roundings and the codes that they
    move, tests/test_gpu_layer_example.py)."""
    for args in (["--steps", "6"], ["--requests", "2", "--beams", "1", "--steps", "3"],
                 ["--requests", "3", "--beams", "8", "--steps", "9", "--vocab", "64", "--layers", "2"]):
        print("[gpu] beam search", args, flush=True)
        assert example.main(args + ["--check"]) < 0.3 * int(args[args.index("--steps") + 1])


@pytest.mark.parametrize("requests,beams,vocab,steps", [(3, 5, 509, 7), (2, 8, 40, 12)])
def test_states_follow_their_sequences(example, requests, beams, vocab, steps):
    """Each best sequence taken through the model again without any reordering: the same states bit for bit, since no
    operator's row depends on where it stands, and scores that add up (a float32 rounding for each
    step, of scores up to 64, and 1e-5 of each log probability)."""
    print("[gpu] beam search, states", requests, beams, vocab, steps, flush=True)
    m = example
    model = m.make_model(2, 256, 8, 64, 128, 2, vocab)
    adapters = m.make_adapters(model, requests, 6)
    adapter = torch.arange(requests, device="cuda", dtype=torch.int32) - 1
    scores, said, states, slots = m.search(model, adapters, adapter, beams, steps)
    own = torch.arange(requests * beams, device="cuda", dtype=torch.int32).view(requests, beams)
    fresh = [torch.zeros_like(s) for s in states]
    tokens = torch.full((requests, beams), m.START, device="cuda")
    total = torch.zeros(requests * beams, dtype=torch.float64, device="cuda")
    over = torch.zeros(requests * beams, dtype=torch.bool, device="cuda")
    for t in range(steps):
        logits = m.step(model, adapters, fresh, own, tokens, adapter)
        tokens = said[:, :, t]
        gained = ssu.token_logprobs(logits.view(requests * beams, vocab), tokens.flatten()).logprob
        total += torch.where(over, 0.0, gained.double())
        over |= tokens.flatten() == m.END
    assert torch.equal(slots.sort(-1).values, own)
    for a, b in zip(states, fresh):
        assert torch.equal(a[slots.flatten().long()], b)
    assert (scores.flatten().double() - total).abs().max() <= steps * (2.0 ** -18 + 1e-4)
    assert len({tuple(s) for s in said[0].tolist()}) == beams  # different sequences
