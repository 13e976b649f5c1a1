"""Workspaces of mx_linear, token_logprobs and ssd_combined_fwd_varlen: a captured graph owns what it writes to, whatever else is
captured, called or allocated on its stream, and an eager call leaves nothing behind.

Every answer is compared bit for bit with that of an eager call on the default stream: the
operators repeat exactly."""
import pytest
import torch

import mamba_selective_state_amd as ssu
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def say(*a):
    print("[gpu] workspaces", *a, flush=True)


class Linear:
    """40 rows of floats: codes and scales go through the workspace."""

    def __init__(self, seed, rows=40):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(rows, 1024, generator=g).bfloat16().cuda()
        self.w, self.ws = ssu.mx_quantize(torch.randn(520, 1024, generator=g).cuda())

    def call(self):
        return (ssu.mx_linear(self.x, self.w, self.ws),)

    def larger(self):
        return Linear(99, 3000).call()

    def change(self, seed):
        self.x.copy_(torch.randn(self.x.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())


class Logprobs:
    """Two rows: each is split over workgroups that leave shares and draw tickets."""

    def __init__(self, seed, rows=2, vocab=60000):
        g = torch.Generator().manual_seed(seed)
        self.logits = (3 * torch.randn(rows, vocab, generator=g)).bfloat16().cuda()
        self.tokens = torch.randint(0, vocab, (rows,), generator=g).cuda()

    def call(self):
        return ssu.token_logprobs(self.logits, self.tokens, 9)

    def larger(self):
        return Logprobs(99, 200, 9000).call()

    def change(self, seed):
        self.logits.copy_((3 * torch.randn(self.logits.shape, generator=torch.Generator().manual_seed(seed))).bfloat16())


class Ssd:
    """A prefill of three sequences: every chunk's state goes through the workspace."""

    def __init__(self, seed, lengths=(300, 17, 129)):
        c = W.ssd(seed=seed, lengths=lengths, heads=8, dim=64, dstate=128, groups=2, chunk_size=128, io="f32",
                  state_dtype="f32")
        self.t = {k: torch.from_numpy(c[k]).cuda() for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")}
        for k in ("x", "B", "C"):
            self.t[k] = self.t[k].bfloat16()
        self.t.update({k: torch.as_tensor(c[k]).cuda() for k in ("cu_seqlens", "cu_chunk_seqlens", "last_chunk_indices", "seq_idx")})
        self.t.update(chunk_size=c["chunk_size"], dt_softplus=True, state_dtype=torch.float32)

    def call(self):
        y = torch.empty_like(self.t["x"])
        return y, ssu.ssd_combined_fwd_varlen(out=y, **self.t)

    def larger(self):
        return Ssd(99, (3000, 500)).call()

    def change(self, seed):
        self.t["x"].copy_(torch.randn(self.t["x"].shape, generator=torch.Generator().manual_seed(seed)).bfloat16())


OPS = pytest.mark.parametrize("Op", [Linear, Logprobs, Ssd])


def expect(op):
    """The answer of an eager call on the default stream."""
    torch.cuda.synchronize()
    r = [t.clone() for t in op.call()]
    torch.cuda.synchronize()
    return r


def same(got, want):
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def replay(graph, out, op, want=None):
    want = expect(op) if want is None else want
    for t in out:
        t.fill_(7)  # an output that a replay does not write shows
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    same(out, want)


@OPS
def test_two_graphs_of_one_capture_stream_in_reverse_order(Op):
    """torch.cuda.graph without a stream captures on one and the same stream; nothing has run there."""
    say(Op.__name__, "two graphs, the second one first")
    ops = [Op(1), Op(2)]
    want = [expect(op) for op in ops]
    graphs, outs = [], []
    for op in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(op.call())
        graphs.append(g)
    for i in (1, 0, 1, 1, 0):
        replay(graphs[i], outs[i], ops[i], want[i])
    for i in (0, 1, 0):
        ops[i].change(50 + i)
        replay(graphs[i], outs[i], ops[i])


@OPS
def test_eager_call_on_the_capture_stream_before_a_replay(Op):
    say(Op.__name__, "eager on the capture stream")
    op, s = Op(3), torch.cuda.Stream()
    want = expect(op)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = op.call()
    with torch.cuda.stream(s):
        for _ in range(3):
            same(op.call(), want)
    torch.cuda.synchronize()
    replay(g, out, op, want)


@OPS
def test_larger_call_between_capture_and_replay(Op):
    """A larger call on the stream of a graph, and memory allocated and filled behind it."""
    say(Op.__name__, "larger call between")
    op, s = Op(4), torch.cuda.Stream()
    want = expect(op)
    with torch.cuda.stream(s):
        op.call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = op.call()
        op.larger()
        s.synchronize()
        # whatever the stream has given back: filled, and looked at after the replays
        filled = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in (2048, 4096, 50000, 200000, 1 << 20, 3 << 20) for _ in range(8)]
    for _ in range(3):
        replay(g, out, op, want)
    assert all(bool((f == 3).all()) for f in filled)
    with torch.cuda.stream(s):
        same(op.call(), want)
    torch.cuda.synchronize()


@OPS
def test_graphs_of_one_capture_stream_replayed_together(Op):
    """Captured on one stream, replayed on two."""
    say(Op.__name__, "two graphs on two streams")
    ops = [Op(5), Op(6)]
    want = [expect(op) for op in ops]
    graphs, outs = [], []
    for op in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([op.call() for _ in range(8)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i, calls in enumerate(outs):
        for out in calls:
            same(out, want[i])


@OPS
def test_graph_outlives_the_one_before_it(Op):
    """The first graph of a capture stream, and its memory, go; the second one still answers."""
    say(Op.__name__, "first graph released")
    ops = [Op(7), Op(8)]
    want = [expect(op) for op in ops]
    graphs, outs = [], []
    for op in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(op.call())
        graphs.append(g)
    replay(graphs[0], outs[0], ops[0], want[0])
    graphs[0].reset()
    del graphs[0], outs[0]
    torch.cuda.empty_cache()
    filled = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in (2048, 50000, 200000, 1 << 20) for _ in range(8)]
    for _ in range(3):
        replay(graphs[0], outs[0], ops[1], want[1])
    assert all(bool((f == 3).all()) for f in filled)


def test_linear_keeps_no_memory():
    """What a product used for its activations is free again after it."""
    say("memory after a product")
    op = Linear(9, 4000)
    op.call()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = op.call()[0]
    torch.cuda.synchronize()
    del y
    assert torch.cuda.memory_allocated() == before
