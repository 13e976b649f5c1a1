"""token_logprobs against its definition in float64 (layer_ref.logprobs).

Ranks and tokens are exact. A log probability is off by the rounding of
(l - m) / temperature (|l - m| < 128 here: below 2^-16), and the sum's relative error
(up to 512 additions a lane: 2^-15); the entropy by the same twice:
ATOL = 1e-4, and 1e-6 of the value."""
import math

import pytest
import torch

import layer_ref as R
import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ATOL, RTOL = 1e-4, 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def say(*a):
    print(*a, flush=True)


def near(got, want):
    got = got.cpu().double()
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.sign() * math.inf, want)  # what float32 holds
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert (same | ((got - want).abs() <= ATOL + RTOL * want.abs())).all(), (got, want)


def check(logits, tokens, top=0, mask=None, temperature=None, **kw):
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    say("[gpu] logprobs", tuple(logits.shape), logits.dtype, "top", top, "mask", mask is not None)
    r = ssu.token_logprobs(d(logits), d(tokens), top=top, mask=d(mask), temperature=d(temperature))
    torch.cuda.synchronize()
    compare(r, logits, tokens, top, mask, temperature)
    return r


def compare(r, logits, tokens, top=0, mask=None, temperature=None):
    ref = R.logprobs(logits, tokens, top, mask, temperature)
    assert torch.equal(r.rank.cpu(), ref["rank"]), (r.rank, ref["rank"])
    near(r.logprob, ref["logprob"])
    near(r.entropy, ref["entropy"])
    if top:
        assert torch.equal(r.top_tokens.cpu(), ref["top_tokens"]), (r.top_tokens, ref["top_tokens"])
        near(r.top_logprobs, ref["top_logprobs"])
    else:
        assert r.top_tokens is None and r.top_logprobs is None


def case(rows, vocab, dt, seed=0, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(rows, vocab, generator=g) * scale).to(DT[dt])
    return logits, torch.randint(0, vocab, (rows,), generator=g)


def bitmask(allow):
    rows, vocab = allow.shape
    words = -(-vocab // 32)
    b = torch.zeros(rows, words * 32, dtype=torch.int64)
    b[:, :vocab] = allow
    w = (b.view(rows, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


VOCABS = [1, 2, 7, 8, 31, 32, 33, 63, 64, 65, 257, 511, 512, 513, 1000, 2047, 2048, 2049, 4095, 4097, 8191, 8193, 10007, 16384,
          33333, 65536, 65537, 131071]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_vocabularies(vocab, dt):
    logits, tokens = case(3, vocab, dt, seed=vocab)
    tokens[0], tokens[1] = 0, vocab - 1
    check(logits, tokens, top=min(32, 5 + vocab % 28))


@pytest.mark.parametrize("rows", [1, 2, 16, 100, 600, 1100, 2300])
@pytest.mark.parametrize("top", [0, 1, 8, 32])
def test_row_counts(rows, top):
    logits, tokens = case(rows, 700, "bf16", seed=rows)
    check(logits, tokens, top=top)


@pytest.mark.parametrize("top", [0, 1, 2, 16, 31, 32])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [20, 1031, 40001])
def test_ties(top, dt, vocab):
    """Few distinct values: alternatives and ranks go by the lowest index."""
    g = torch.Generator().manual_seed(top)
    for distinct in (1, 2, 5):
        logits = torch.randint(0, distinct, (4, vocab), generator=g).to(DT[dt])
        logits[logits == 0] = -0.0  # and -0 is 0
        logits[:, ::3] = torch.where(logits[:, ::3] == 0, torch.zeros(()).to(DT[dt]), logits[:, ::3])
        tokens = torch.randint(0, vocab, (4,), generator=g)
        check(logits, tokens, top=top)


@pytest.mark.parametrize("order", ["up", "down"])
@pytest.mark.parametrize("rows", [1, 1030])
def test_sorted_logits(order, rows):
    """Every logit better than all before it, and the other way round."""
    v = 5000
    l = torch.arange(v).float() / 50
    l = l if order == "up" else l.flip(0)
    logits = l.repeat(rows, 1)
    check(logits, torch.full((rows,), v // 3), top=32)


@pytest.mark.parametrize("rows", [3, 1040])
@pytest.mark.parametrize("vocab", [33, 4096, 50021])
def test_mask_and_temperature(rows, vocab):
    if rows * vocab > 10 ** 7:
        rows = 150
    g = torch.Generator().manual_seed(vocab)
    logits, tokens = case(rows, vocab, "f32", seed=vocab)
    logits[torch.rand(rows, vocab, generator=g) < 0.1] = -math.inf
    allow = torch.rand(rows, vocab, generator=g) < torch.tensor([0.9, 0.5, 0.01])[torch.arange(rows) % 3][:, None]
    allow[0] = False                       # nothing left
    allow[1] = False
    allow[1, vocab // 2] = True            # one token left
    logits[1, vocab // 2] = 0.5
    tokens[1] = vocab // 2
    # what masked places hold does not matter
    junk = torch.tensor([math.nan, math.inf, torch.finfo(torch.float32).max, torch.finfo(torch.float32).min])
    logits = torch.where(allow, logits, junk[torch.randint(0, 4, (rows, vocab), generator=g)])
    temperature = 0.3 + torch.rand(rows, generator=g)
    mask = bitmask(allow)
    r = check(logits, tokens, 7, mask, temperature)
    assert float(r.logprob[0]) == -math.inf and float(r.entropy[0]) == 0 and int(r.rank[0]) == -1
    assert float(r.logprob[1]) == 0 and int(r.rank[1]) == 0 and r.top_tokens[1].tolist()[1:] == [-1] * 6
    # one mask shared by all rows
    one = ssu.token_logprobs(logits.cuda(), tokens.cuda(), 7, mask[2:3].cuda(), temperature.cuda())
    compare(one, logits, tokens, 7, mask[2:3].expand(rows, -1), temperature)


def test_special_logits():
    v = 3000
    logits, tokens = case(9, v, "f32", seed=4)
    logits[0, 17] = math.nan
    logits[1, 2999] = math.inf
    logits[2] = -math.inf                                  # nothing left
    logits[3] = torch.finfo(torch.float32).min             # the lowest value is a logit like any other
    logits[4] = -math.inf
    logits[4, 7] = torch.finfo(torch.float32).min
    tokens[4] = 7
    logits[5, int(tokens[5])] = -math.inf
    tokens[6], tokens[7] = -1, v                           # outside
    logits[8] = -1e30
    logits[8, 5] = 1e30
    check(logits, tokens, top=4)


def test_bad_temperature():
    logits, tokens = case(4, 100, "bf16")
    check(logits, tokens, top=2, temperature=torch.tensor([1.0, 0.0, -1.0, math.nan]))


def test_peaked_and_flat():
    """Entropy at both ends: near 0, and log(vocab) exactly."""
    logits = torch.zeros(2, 20000)
    logits[0, 123] = 60
    r = check(logits, torch.tensor([123, 5]), top=3)
    assert abs(float(r.entropy[1]) - math.log(20000)) < 1e-5 and abs(float(r.entropy[0])) < 1e-6


def test_strides_and_index_types():
    logits, tokens = case(5, 2000, "f16", seed=8)
    wide = torch.full((5, 2103), math.nan, dtype=torch.float16, device="cuda")
    wide[:, 1:2001] = logits.cuda()
    pairs = torch.stack((tokens, tokens + 1), 1).cuda()
    temps = torch.stack((torch.full((5,), 0.7), torch.full((5,), -1.0)), 1).cuda()
    words = bitmask(torch.rand(5, 2000) < 0.5)
    wmask = torch.zeros(5, 70, dtype=torch.int32, device="cuda")
    wmask[:, 3:66] = words.cuda()
    for t in (pairs[:, 0], pairs.int()[:, 0]):
        r = ssu.token_logprobs(wide[:, 1:2001], t, 6, wmask[:, 3:66], temps[:, 0])
        compare(r, logits, tokens, 6, words, torch.full((5,), 0.7))
    row = ssu.token_logprobs(logits[:1].cuda().expand(4, -1), tokens[:1].cuda().expand(4), 2)
    compare(row, logits[:1].expand(4, -1), tokens[:1].expand(4), 2)


def test_offsets_beyond_32_bits():
    stride = 1_500_000_001
    logits, tokens = case(3, 700, "bf16", seed=2)
    big = torch.empty(2 * stride + 800, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 700), (stride, 1))
    x.copy_(logits.cuda())
    say("[gpu] logprobs, rows %d elements apart" % stride)
    compare(ssu.token_logprobs(x, tokens.cuda(), 3), logits, tokens, 3)


def test_repeated_calls_streams_and_graph():
    """The same answer from the same inputs, bit for bit, on any stream, after calls of
    other sizes, and from a replayed graph."""
    logits, tokens = (t.cuda() for t in case(2, 60000, "bf16", seed=3))
    other, ot = (t.cuda() for t in case(40, 9000, "f32", seed=5))
    want = ssu.token_logprobs(logits, tokens, 9)
    compare(want, logits.cpu(), tokens.cpu(), 9)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            for _ in range(4):
                ssu.token_logprobs(other, ot, 20)
                got.append(ssu.token_logprobs(logits, tokens, 9))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ssu.token_logprobs(logits, tokens, 9)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            r = ssu.token_logprobs(logits, tokens, 9)
    for i in range(4):
        logits.copy_(case(2, 60000, "bf16", seed=10 + i)[0].cuda())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, ssu.token_logprobs(logits, tokens, 9)))


def test_empty():
    r = ssu.token_logprobs(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), 3)
    assert r.logprob.shape == (0,) and r.top_tokens.shape == (0, 3)
    r = ssu.token_logprobs(torch.empty(2, 0, device="cuda"), torch.tensor([0, -1], device="cuda"), 2)
    assert r.logprob.tolist() == [-math.inf] * 2 and r.rank.tolist() == [-1, -1] and r.top_tokens.tolist() == [[-1, -1]] * 2
