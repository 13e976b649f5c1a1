"""token_logprobs where one token holds nearly all of the probability: the digits of what is left.

A row's logits (over the temperature) are 0 for one token, -gap for another one and -60 for the rest, whose
e^-60 leave the sum alone. The sum is then 1 + e^-gap, rounded where the two meet (2^-24) and
once for each join with a sum of other references (c times 1: nothing); (x - m) / T of the peak is 0. With
e^-gap good to 2^-19 of itself (its exponent, below 24, is a product with two rounded factors, and the
exponential within an ulp) log s is good to TOL = 2^-23 for gap >= 8: 2^-24 from the sum, e^-8 2^-19 from the
term, the logarithm's ulp. The entropy is log s + gap e^-gap / s: twice that. The second token's
value -gap - log s has four roundings of gap: 2^-22 of it."""
import math

import pytest
import torch

import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def log_s(gap):
    return math.log1p(math.exp(-gap))


@pytest.mark.parametrize("gap", [8.0, 9.5, 10.75, 11.0, 11.25, 14.0])
@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("temperature", [None, 0.25, 3.0])
def test_peak(gap, rows, temperature):
    vocab, temp = 20000, temperature or 1.0
    print("[gpu] peak", gap, rows, temperature, flush=True)
    # the second token before the peak, so that it is what the peak is first compared with; in the
    # same access, another wave's, the last one, another workgroup's
    for second, peak in ((3, 5), (3, 700), (100, 19999), (1030, 2 * 2048 + 1030), (9000, 19000), (19000, 40)):
        logits = torch.full((rows, vocab), -60.0 * temp)
        logits[:, second], logits[:, peak] = -gap * temp, 0.0
        logits += 4.0  # exact: every value is a quarter of a small number
        t = None if temperature is None else torch.full((rows,), temp, device="cuda")
        r = ssu.token_logprobs(logits.cuda(), torch.full((rows,), peak, device="cuda"), 2, temperature=t)
        s = log_s(gap)
        entropy = s + gap * math.exp(-gap) / (1 + math.exp(-gap))
        assert (r.rank == 0).all() and r.top_tokens[0].tolist() == [peak, second]
        assert float((r.logprob.double() + s).abs().max()) <= TOL, (second, peak)
        assert float((r.top_logprobs[:, 0].double() + s).abs().max()) <= TOL, (second, peak)
        assert float((r.entropy.double() - entropy).abs().max()) <= 2 * TOL, (second, peak)
        assert float((r.top_logprobs[:, 1].double() + gap + s).abs().max()) <= TOL + gap * 2.0 ** -22, (second, peak)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rising_peaks(dt):
    """Each access's largest logit a little above all before it: the last one's reference holds."""
    vocab = 64 * 512
    logits = torch.full((260, vocab), -80.0)
    logits[:, 7::512] = torch.arange(64).float() / 2
    logits = logits.to(dt)
    l = logits[:1].double()
    want = torch.log_softmax(l, -1)
    print("[gpu] rising peaks", dt, flush=True)
    tokens = torch.full((260,), 63 * 512 + 7, device="cuda")
    r = ssu.token_logprobs(logits.cuda(), tokens, 3)
    # log s = 0.93: 64 terms, each within 2^-19 of itself, and as many sums within 2^-24 of theirs
    tol = 2.0 ** -19 + 64 * 2.0 ** -24
    assert float((r.logprob.cpu().double() - want[0, 63 * 512 + 7]).abs().max()) <= tol
    assert float((r.entropy.cpu().double() + (want.exp() * want).sum()).abs().max()) <= 4 * tol
    assert (r.rank == 0).all() and r.top_tokens[5].tolist() == [63 * 512 + 7, 62 * 512 + 7, 61 * 512 + 7]
