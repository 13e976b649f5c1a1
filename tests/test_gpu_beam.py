"""beam_select against its definition in float64 (search_ref).

A score is off by the rounding to float32, and by what the float32 sum of exponentials is off: a lane
adds vocab / 2048 terms of eight, the wave and the workgroup 8 more, each addition by 2^-24 of the sum at most, and an
exponential is off by 2^-21 (its argument's rounding and the instruction's). Parents and tokens are those of the
definition, but where two beams' continuations are nearer to each other than twice that."""
import math

import pytest
import torch

import mamba_selective_state_amd as ssu
import search_ref as S

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def say(*a):
    print("[gpu] beam_select", *a, flush=True)


def inputs(batch, beams, vocab, dt, seed=0, mask=None, ended=False):
    g = torch.Generator().manual_seed(seed)
    x = 3 * torch.randn(batch * beams, vocab, generator=g)
    x[torch.rand(x.shape, generator=g) < 0.02] = -math.inf
    c = {"logits": x.to(DT[dt]), "scores": -10 * torch.rand(batch, beams, generator=g), "finished": None, "mask": None}
    if ended:
        c["finished"] = torch.rand(batch, beams, generator=g) < 0.25
        c["scores"][torch.rand(batch, beams, generator=g) < 0.25] = -math.inf
    if mask is not None:
        bits = torch.rand(batch * beams if mask == "rows" else 1, -(-vocab // 32), 32, generator=g) < 0.5
        bits[:1] &= torch.rand(1, generator=g) < 0.5  # at times a row that allows nothing
        w = (bits.long() << torch.arange(32)).sum(-1)
        c["mask"] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    return c


def dev(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def run(c, keep, **kw):
    d = dev(c)
    say(tuple(c["logits"].shape), c["logits"].dtype, "scores", tuple(c["scores"].shape), "keep", keep)
    r = ssu.beam_select(d["logits"], d["scores"], keep, finished=d["finished"], mask=d["mask"], **kw)
    torch.cuda.synchronize()
    return ssu.BeamSelection(*(t.cpu() for t in r))


def off(vocab):
    return (vocab / 2048 + 8) * 2.0 ** -24 + 2.0 ** -21


def check(r, c, keep, end_token=0):
    e = off(c["logits"].shape[-1])
    every = S.scores_of(c["logits"], c["scores"], c["finished"], end_token, c["mask"])
    want = S.beam_select(c["logits"], c["scores"], keep, c["finished"], end_token, c["mask"])
    for b, found in enumerate(every):
        if found is None:
            assert torch.isnan(r.scores[b]).all() and (r.parents[b] == -1).all() and (r.tokens[b] == -1).all()
            continue
        of = {(i, t): s for s, i, t, _ in found}
        n = min(keep, len(found))
        assert (r.parents[b, n:] == -1).all() and (r.tokens[b, n:] == -1).all() and (r.scores[b, n:] == -math.inf).all()
        got = list(zip(r.parents[b, :n].tolist(), r.tokens[b, :n].tolist()))
        assert len(set(got)) == n and all(q in of for q in got), (b, got)
        for at, q in enumerate(got):
            best = float(want[0][b, at])
            assert abs(of[q] - best) <= 2 * e, (b, at, q, of[q], best)
            assert abs(float(r.scores[b, at]) - of[q]) <= e + 2.0 ** -24 * abs(of[q]), (b, at)
            if q != (int(want[1][b, at]), int(want[2][b, at])):
                # another one only if it is as near, and of another beam
                assert q[0] != int(want[1][b, at]), (b, at, q)


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 511, 512, 513, 2047, 2049, 4096, 8200, 33000])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_vocabularies(vocab, dt):
    c = inputs(3, 4, vocab, dt, seed=vocab)
    check(run(c, 8), c, 8)


@pytest.mark.parametrize("batch,beams", [(1, 1), (1, 2), (1, 64), (2, 17), (5, 64), (70, 4), (300, 1), (33, 8)])
@pytest.mark.parametrize("keep", [1, 2, 16, 31, 32])
def test_beams_and_keep(batch, beams, keep):
    c = inputs(batch, beams, 700, "f32", seed=batch + beams + keep)
    check(run(c, keep), c, keep)


def test_large_batch():
    c = inputs(1500, 4, 33, "f16", seed=8, ended=True)
    check(run(c, 8, end_token=3), c, 8, 3)


@pytest.mark.parametrize("mask", [None, "one", "rows"])
@pytest.mark.parametrize("vocab", [5, 100, 3001])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_masks_and_ended_beams(mask, vocab, dt):
    for seed in range(4):
        c = inputs(6, 5, vocab, dt, seed=seed, mask=mask, ended=True)
        check(run(c, 10, end_token=vocab - 1), c, 10, vocab - 1)


def test_one_live_beam():
    """A search's first step: all beams but the first at -inf."""
    for beams in (2, 8, 64):
        c = inputs(2, beams, 5000, "f32", seed=beams)
        c["scores"][:, 1:] = -math.inf
        c["scores"][:, 0] = 0
        check(run(c, 16), c, 16)


def test_nothing_left():
    c = inputs(3, 4, 100, "f32")
    c["scores"][0] = -math.inf
    c["logits"][4:8] = -math.inf
    c["finished"] = torch.zeros(3, 4, dtype=torch.uint8)
    c["finished"][2] = 7  # any value but 0
    c["scores"][2] = torch.tensor([-3.0, -1.0, -math.inf, -2.0])
    r = run(c, 6, end_token=9)
    check(r, c, 6, 9)
    assert r.parents[2].tolist() == [1, 3, 0, -1, -1, -1] and r.tokens[2].tolist() == [9, 9, 9, -1, -1, -1]
    assert r.scores[2, :3].tolist() == [-1.0, -2.0, -3.0]


def test_nan_and_infinity():
    """They spoil their own request; in beams that are not read, and behind a mask, they change nothing."""
    c = inputs(7, 3, 600, "f32")
    c["finished"] = torch.zeros(7, 3, dtype=torch.bool)
    c["mask"] = torch.full((21, 19), -1, dtype=torch.int32)
    c["logits"][1, 77] = math.nan
    c["logits"][5, 3] = math.inf
    c["scores"][2, 1] = math.nan
    c["scores"][3, 0] = math.inf
    c["logits"][13] = math.nan
    c["scores"][4, 1] = -math.inf
    c["logits"][16] = math.inf
    c["finished"][5, 1] = True
    c["logits"][19, 64:96] = math.nan
    c["mask"][19, 2] = 0
    r = run(c, 5, end_token=4)
    check(r, c, 5, 4)
    bad = torch.isnan(r.scores).all(-1).tolist()
    assert bad == [True, True, True, True, False, False, False]
    c["finished"][6, 0] = True
    c["scores"][6, 0] = math.nan  # of an ended beam too
    assert torch.isnan(run(c, 5, end_token=4).scores[6]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [40, 6000])
def test_equal_scores(vocab, dt):
    """Equal beams and equal logits: by beam, then by token, exactly."""
    g = torch.Generator().manual_seed(vocab)
    row = torch.randint(-3, 4, (1, vocab), generator=g).to(DT[dt])
    c = {"logits": row.expand(8, vocab).contiguous(), "scores": torch.full((2, 4), -1.5), "finished": None, "mask": None}
    r = run(c, 32)
    want = S.beam_select(c["logits"], c["scores"], 32)
    assert torch.equal(r.parents, want[1]) and torch.equal(r.tokens, want[2])
    c["logits"] = torch.zeros(8, vocab, dtype=DT[dt])
    c["logits"][:, ::2] = -0.0  # equal to 0
    r = run(c, 32)
    assert r.parents.tolist() == [[0] * 32] * 2 and r.tokens.tolist() == [list(range(32))] * 2


@pytest.mark.parametrize("beams", [3, 64])
def test_all_equal(beams):
    """More equal scores than the second kernel has room for: 64 beams of many shares each."""
    d = torch.zeros(beams, 40000, dtype=torch.bfloat16, device="cuda")
    say("all equal", beams)
    r = ssu.beam_select(d, torch.zeros(1, beams, device="cuda"), 32)
    assert r.parents.tolist() == [[0] * 32] and r.tokens.tolist() == [list(range(32))]
    assert torch.allclose(r.scores.cpu(), torch.full((1, 32), -math.log(40000)), atol=1e-5)
    # Beams in pairs of equal scores, one token each that stands out: it scores 5 - i // 2 - L, L = log(39999 + e^5), and beam 0's
    # and 1's other tokens score -L. So the first ten (fewer where there are fewer beams) are known, and all that follow
    # score -L, whichever of equal ones they are.
    at = torch.randint(0, 40000, (beams,), generator=torch.Generator().manual_seed(beams))
    d[torch.arange(beams), at] = 5
    scores = -(torch.arange(beams) // 2).float()[None]
    n, first = min(32, beams), min(10, beams)
    r = ssu.beam_select(d, scores.cuda(), n)
    assert r.parents[0, :first].tolist() == list(range(first))
    assert torch.equal(r.tokens[0, :first].cpu().long(), at[:first])
    want = torch.tensor([max(5 - i // 2, 0) for i in range(n)]) - math.log(39999 + math.exp(5))
    assert torch.allclose(r.scores[0].cpu(), want, atol=1e-5)


def test_shapes_that_do_not_agree():
    x = torch.zeros(3, 4, 50, device="cuda")
    for logits, scores in ((x, (4, 3)), (x, (12, 1)), (x.view(1, 3, 4, 50), (3, 4)), (x.view(12, 50), (3, 5))):
        with pytest.raises(ValueError):
            ssu.beam_select(logits, torch.zeros(scores, device="cuda"), 2)


def test_extreme_logits():
    c = inputs(2, 2, 1500, "f32")
    c["logits"][0] = -3e38
    c["logits"][0, 700:710] = 3e38
    c["logits"][1] = torch.linspace(-1e30, 1e30, 1500)
    c["logits"][2] *= 1e-30
    r = run(c, 12)
    assert r.parents[0].tolist().count(0) + r.parents[0].tolist().count(1) == 12
    # ten equal logits hold all of beam 0; of beam 1 the largest one does
    assert abs(float(r.scores[0][r.parents[0] == 0][0]) - (float(c["scores"][0, 0]) - math.log(10))) < 1e-5
    assert sorted(r.tokens[0][r.parents[0] == 0].tolist())[:10] == list(range(700, 710))
    assert int(r.tokens[0][r.parents[0] == 1][0]) == 1499
    check(run({k: v[2:] if k == "logits" else v[1:] if k == "scores" else v for k, v in c.items()}, 12),
          {k: v[2:] if k == "logits" else v[1:] if k == "scores" else v for k, v in c.items()}, 12)


def test_strides_and_dimensions():
    c = inputs(4, 3, 777, "f16", seed=3, mask="rows", ended=True)
    want = run(c, 9)
    check(want, c, 9)
    d = dev(c)
    wide = torch.full((12, 1001), 60000.0, dtype=torch.float16, device="cuda")
    wide[:, 3:780] = d["logits"]
    scores = torch.empty(3, 4, device="cuda").t()
    scores.copy_(d["scores"])
    finished = torch.zeros(4, 6, dtype=torch.bool, device="cuda")[:, ::2]
    finished.copy_(d["finished"])
    for logits, mask in ((wide[:, 3:780], d["mask"]), (d["logits"].view(4, 3, 777), d["mask"].view(4, 3, -1))):
        r = ssu.beam_select(logits, scores, 9, finished=finished, mask=mask)
        for a, b in zip(r, want):
            assert torch.equal(a.cpu(), b)


def test_repeats_streams_and_graph():
    c = inputs(3, 5, 40000, "bf16", seed=5, ended=True)
    want = run(c, 10)
    d = dev(c)

    def call():
        return ssu.beam_select(d["logits"], d["scores"], 10, finished=d["finished"])
    for _ in range(3):
        for a, b in zip(call(), want):
            assert torch.equal(a.cpu(), b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = call()
    s.synchronize()
    for a, b in zip(r, want):
        assert torch.equal(a.cpu(), b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = call()
    for i in range(4):
        d["logits"].copy_(inputs(3, 5, 40000, "bf16", seed=20 + i)["logits"].cuda())
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(r, call()):
            assert torch.equal(a, b) or (torch.isnan(a).all() and torch.isnan(b).all())


def test_offsets_beyond_32_bits():
    """Rows 1.2e9 elements apart."""
    stride = 1_200_000_007
    c = inputs(1, 3, 900, "bf16", seed=9)
    big = torch.empty(2 * stride + 1024, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 900), (stride, 1), 5)
    x.copy_(c["logits"].cuda())
    say("rows %d elements apart" % stride)
    r = ssu.beam_select(x, c["scores"].cuda(), 6)
    check(ssu.BeamSelection(*(t.cpu() for t in r)), c, 6)


def test_empty():
    z = ssu.beam_select(torch.empty(0, 50, device="cuda"), torch.empty(0, 4, device="cuda"), 3)
    assert z.scores.shape == (0, 3) and z.tokens.dtype == torch.int32
    z = ssu.beam_select(torch.randn(4, 50, device="cuda"), torch.zeros(1, 4, device="cuda"), 0)
    assert z.parents.shape == (1, 0)
    z = ssu.beam_select(torch.empty(4, 0, device="cuda"), torch.zeros(1, 4, device="cuda"), 2)
    assert z.parents.tolist() == [[-1, -1]] and z.scores.tolist() == [[-math.inf, -math.inf]]
