"""Workspaces of beam_select and add_lora, and reorder_states beside them: captured graphs own what they write to, calls on two
streams do not meet, and the C entry points stay inside the workspace they ask for.

Answers are compared bit for bit with those of an eager call on the default stream."""
import pytest
import torch

import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def say(*a):
    print("[gpu] search workspaces", *a, flush=True)


class Beam:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.logits = (3 * torch.randn(2 * 5, 30000, generator=g)).bfloat16().cuda()
        self.scores = -torch.rand(2, 5, generator=g).cuda()

    def call(self):
        return tuple(ssu.beam_select(self.logits, self.scores, 10))


class Lora:
    """The rows' number decides which kernels run."""

    def __init__(self, seed, rows=90):
        g = torch.Generator().manual_seed(seed)
        self.y = torch.randn(rows, 200, generator=g).bfloat16().cuda()
        self.x = torch.randn(rows, 512, generator=g).bfloat16().cuda()
        self.a = (torch.randn(7, 16, 512, generator=g) / 20).bfloat16().cuda()
        self.b = torch.randn(7, 200, 16, generator=g).bfloat16().cuda()
        self.ids = torch.randint(-1, 7, (rows,), generator=g).int().cuda()

    def call(self):
        out = self.y.clone()
        return (ssu.add_lora(out, self.x, self.a, self.b, self.ids),)


class ManyLora(Lora):
    def __init__(self, seed):
        super().__init__(seed, 700)


class Reorder:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.pool = torch.randn(20, 3000, generator=g).cuda()
        self.slots = torch.randperm(20, generator=g)[:18].view(3, 6).int().cuda()
        self.parents = torch.randint(0, 6, (3, 6), generator=g).int().cuda()

    def call(self):
        pool = self.pool.clone()
        return ssu.reorder_states(pool, self.slots, self.parents), pool


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


KINDS = [Beam, Lora, ManyLora, Reorder]


@pytest.mark.parametrize("kind", KINDS)
def test_two_graphs_of_one_stream(kind):
    """Both captured on one stream, replayed at the same time on two, with eager calls between."""
    say(kind.__name__, "two graphs")
    one, two, other = kind(1), kind(2), kind(3)
    want = one.call(), two.call(), other.call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs, got = [], []
    for c in (one, two):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got.append(c.call())
        graphs.append(g)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        for t in got[0] + got[1]:
            t.zero_()
        torch.cuda.synchronize()
        for g, at in zip(graphs, streams):
            with torch.cuda.stream(at):
                g.replay()
        eager = other.call()
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1]) and same(eager, want[2])


@pytest.mark.parametrize("kind", KINDS)
def test_calls_on_two_streams(kind):
    say(kind.__name__, "two streams")
    cases = [kind(i) for i in range(2)]
    want = [c.call() for c in cases]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(cases[i].call())
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(r, want[i]) for r in got[i])


def guarded(bytes_):
    """A workspace between guard bytes."""
    m = torch.full((bytes_ + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    assert m.data_ptr() % 256 == 0
    return m, m.data_ptr() + 256


def intact(m):
    return bool((m[:256] == 0x5A).all() and (m[-256:] == 0x5A).all())


@pytest.mark.parametrize("rows,adapters,k,n,rank", [(1, 1, 64, 8, 4), (256, 9, 4096, 300, 16), (257, 4096, 256, 72, 64), (3000, 5, 1024, 2000, 128)])
def test_lora_workspace_between_guards(rows, adapters, k, n, rank):
    say("add_lora", rows, adapters, k, n, rank)
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, k, generator=g).bfloat16().cuda()
    a = (torch.randn(adapters, rank, k, generator=g) / 30).bfloat16().cuda()
    b = torch.randn(adapters, n, rank, generator=g).bfloat16().cuda()
    ids = torch.randint(0, adapters, (rows,), generator=g).int().cuda()
    y = torch.randn(rows, n, generator=g).bfloat16().cuda()
    want = ssu.add_lora(y.clone(), x, a, b, ids)
    args = ssu.make_lora_args(y, x, a, b, ids)
    need = ssu.ssu_add_lora_workspace_bytes(args)
    m, at = guarded(need)
    ssu.ssu_add_lora(args, at, need)
    torch.cuda.synchronize()
    assert intact(m) and torch.equal(y, want)


@pytest.mark.parametrize("batch,beams,vocab,keep", [(1, 1, 9, 1), (1, 4, 65536, 8), (1, 64, 70000, 32), (50, 6, 5000, 12)])
def test_beam_workspace_between_guards(batch, beams, vocab, keep):
    say("beam_select", batch, beams, vocab, keep)
    g = torch.Generator().manual_seed(vocab)
    logits = torch.randn(batch * beams, vocab, generator=g).cuda()
    scores = -torch.rand(batch, beams, generator=g).cuda()
    want = ssu.beam_select(logits, scores, keep)
    out = [torch.full((batch, keep), 7, dtype=t.dtype, device="cuda") for t in want]
    args = ssu.make_beam_args(logits, scores, *out)
    need = ssu.ssu_beam_select_workspace_bytes(args)
    m, at = guarded(need)
    ssu.ssu_beam_select(args, at, need)
    torch.cuda.synchronize()
    assert intact(m) and same(out, want)
