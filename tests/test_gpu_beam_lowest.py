"""beam_select on float32 logits at the lowest finite value, which programs write in place of -inf: logits like any
others. Parents and tokens are the definition's exactly: which of equal logits come first is no matter of rounding, and all
others here are far apart. Scores are off by what test_gpu_beam.py allows."""
import math

import pytest
import torch

import mamba_selective_state_amd as ssu
import search_ref as S
from test_gpu_beam import off

pytestmark = pytest.mark.gpu
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def check(logits, scores, keep, mask=None):
    print("[gpu] beam_select, lowest logits", tuple(logits.shape), tuple(scores.shape), keep, mask is not None, flush=True)
    r = ssu.beam_select(logits.cuda(), scores.cuda(), keep, mask=None if mask is None else mask.cuda())
    want = S.beam_select(logits, scores, keep, mask=mask)
    assert torch.equal(r.parents.cpu(), want[1]) and torch.equal(r.tokens.cpu(), want[2])
    some = want[0] > -math.inf
    assert (r.scores.cpu()[~some] == -math.inf).all()
    got = r.scores.cpu().double()[some]
    assert ((got - want[0][some]).abs() <= off(logits.shape[-1]) + 2.0 ** -24 * want[0][some].abs()).all()


def words(bits):
    w = (torch.nn.functional.pad(bits, (0, -bits.shape[1] % 32)).reshape(bits.shape[0], -1, 32).long() << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def ordinary(vocab):
    """Far apart, in the middle of accesses and shares, the larger ones later."""
    at = [vocab * 3 // 7, vocab * 2 // 3, vocab * 5 // 6]
    return at, torch.tensor([-40.0, 1.5, 3.0])


@pytest.mark.parametrize("vocab", [1, 9, 3000, 70000])
@pytest.mark.parametrize("beams,keep", [(1, 1), (1, 8), (3, 32)])
def test_all_lowest(vocab, beams, keep):
    """More equal ones than the list of a share holds, in one share and in several."""
    check(torch.full((2 * beams, vocab), LOWEST), -torch.arange(2.0 * beams).view(2, beams), keep)


@pytest.mark.parametrize("vocab", [40, 3000, 70000])
@pytest.mark.parametrize("beams", [1, 4])
@pytest.mark.parametrize("keep", [2, 8, 32])
def test_fewer_ordinary_logits_than_kept(vocab, beams, keep):
    x = torch.full((beams, vocab), LOWEST)
    at, v = ordinary(vocab)
    x[:, at] = v
    x[:, 5] = -math.inf
    # the best of beam i + 1 stands between two of beam i
    check(x, -0.25 * torch.arange(float(beams))[None], keep)


def test_beams_of_lowest_logits_beside_others():
    x = torch.full((6, 2100), LOWEST)
    at, v = ordinary(2100)
    x[1, at] = v
    x[4] = -math.inf
    x[5, 7:] = -math.inf
    check(x, torch.tensor([[-1.0, -2.5, -math.inf], [-9.0, -1.0, -3.25]]), 20)


@pytest.mark.parametrize("vocab", [50, 3000, 70000])
def test_behind_a_mask(vocab):
    """One allowed token, whose logit is the lowest; a few; half of them; none."""
    x = torch.full((4, vocab), LOWEST)
    at, v = ordinary(vocab)
    x[2:, at] = v
    bits = torch.zeros(4, vocab, dtype=torch.bool)
    bits[0, vocab - 7] = True
    bits[1, vocab // 2::vocab // 8] = True
    bits[2] = torch.rand(vocab, generator=torch.Generator().manual_seed(vocab)) < 0.5
    bits[2, at] = True
    for keep in (1, 8, 32):
        check(x, torch.tensor([[-2.0], [-1.0], [-0.5], [-3.0]]), keep, words(bits))
        check(x, torch.tensor([[-2.0, -1.0, -0.5, -3.0]]), keep, words(bits))
