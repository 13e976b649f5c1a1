"""reorder_states against its definition (search_ref.reorder): whole numbers and copies, so equal bit for
bit, slots that nothing is copied to included."""
import pytest
import torch

import mamba_selective_state_amd as ssu
import search_ref as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def say(*a):
    print("[gpu] reorder_states", *a, flush=True)


def pool(slots, shape, dtype, g):
    if dtype == torch.uint8 or dtype == torch.int32 or dtype == torch.int64:
        return torch.randint(0, 200, (slots, *shape), generator=g).to(dtype)
    return torch.randn((slots, *shape), generator=g).to(dtype)


def inputs(batch, beams, shapes, seed=0, low=0):
    g = torch.Generator().manual_seed(seed)
    n = batch * beams + 2
    slots = torch.randperm(n, generator=g)[:batch * beams].view(batch, beams)
    parents = torch.randint(low, beams, (batch, beams), generator=g)
    return [pool(n, s, t, g) for s, t in shapes], slots, parents


def check(pools, slots, parents, index=torch.int32, want_index=None):
    d = [p.cuda() for p in pools]
    out = ssu.reorder_states(d, slots.to(index).cuda(), parents.to(index).cuda())
    torch.cuda.synchronize()
    want, new = S.reorder(pools, slots, parents)
    assert out.dtype == index and torch.equal(out.cpu().long(), new)
    for a, b in zip(d, want):
        assert torch.equal(a.cpu(), b)


SHAPES = [([((5,), torch.float32)]), ([((1,), torch.uint8)]), ([((17,), torch.uint8), ((3, 7, 11), torch.bfloat16)]),
          ([((4, 64, 128), torch.float32), ((320, 3), torch.bfloat16)]), ([((16383,), torch.uint8), ((16385,), torch.uint8)]),
          ([((9, 5), torch.float64), ((33,), torch.int64), ((2, 2, 2, 2), torch.float16)]), ([((70001,), torch.float16)])]


@pytest.mark.parametrize("shapes", SHAPES, ids=range(len(SHAPES)))
@pytest.mark.parametrize("batch,beams", [(1, 1), (1, 4), (3, 5), (9, 8)])
def test_shapes(shapes, batch, beams):
    say(batch, beams, shapes)
    for seed in range(3):
        check(*inputs(batch, beams, shapes, seed=seed, low=-1))


@pytest.mark.parametrize("beams", [1, 2, 3, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_beams(beams, index):
    say(beams, index)
    for seed in range(4):
        check(*inputs(5, beams, [((40,), torch.float32)], seed=seed, low=-2), index=index)


def test_patterns():
    """All from one beam, the same order, reversed, none."""
    pools, slots, _ = inputs(4, 8, [((100,), torch.bfloat16)])
    parents = torch.stack((torch.full((8,), 5), torch.arange(8), torch.arange(8).flip(0), torch.full((8,), -1)))
    say("patterns")
    check(pools, slots, parents)


def test_numbers_out_of_range():
    """Parents outside the beams count as none; slots that the pools do not have are not copied from or to."""
    pools, slots, parents = inputs(6, 4, [((50,), torch.float32), ((6,), torch.uint8)], seed=3)
    pools[1] = pools[1][:20]  # a shorter pool
    slots[0, 1], slots[1, 2], slots[2, 0] = -1, 10 ** 6, 2 ** 40
    parents[0] = torch.tensor([1, 1, 0, 1])
    parents[1] = torch.tensor([0, 0, 0, 0])
    parents[2] = torch.tensor([0, 0, 3, 3])
    parents[3] = torch.tensor([4, -7, 2 ** 40, 2])
    say("numbers out of range")
    check(pools, slots, parents, index=torch.int64)


def test_large_batch():
    say("3000 requests")
    check(*inputs(3000, 3, [((5, 3), torch.bfloat16)], seed=12, low=-1))


def test_many_pools():
    """More than one launch takes."""
    pools, slots, parents = inputs(2, 4, [((i + 1,), torch.uint8) for i in range(150)], seed=4)
    say("150 pools")
    check(pools, slots, parents)


def test_no_pools_and_empty_ones():
    slots, parents = torch.tensor([[3, 1, 2]]), torch.tensor([[2, 2, 0]])
    for pools in ([], [torch.empty(5, 0, device="cuda")], torch.empty(5, 3, 0, device="cuda")):
        out = ssu.reorder_states(pools, slots.cuda(), parents.cuda())
        assert out.tolist() == [[2, 1, 3]]
    p = torch.ones(4, 3, device="cuda")
    out = ssu.reorder_states(p, torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 3) and (p == 1).all()


def test_strided_pools_slots_and_out():
    """Slots apart from each other, off any alignment; tables as views; a given output of other width."""
    pools, slots, parents = inputs(3, 4, [((130,), torch.uint8)], seed=6)
    want, new = S.reorder(pools, slots, parents)
    wide = torch.full((14, 211), 9, dtype=torch.uint8, device="cuda")
    wide[:, 7:137] = pools[0].cuda()
    ts = torch.empty(4, 3, dtype=torch.int64, device="cuda").t()
    ts.copy_(slots)
    tp = torch.zeros(3, 8, dtype=torch.int32, device="cuda")[:, ::2]
    tp.copy_(parents)
    out = torch.full((3, 9), -5, dtype=torch.int32, device="cuda")
    say("strided")
    r = ssu.reorder_states(wide[:, 7:137], ts, tp, out_slots=out[:, 2:6])
    assert r.data_ptr() == out[:, 2:6].data_ptr()
    assert torch.equal(out[:, 2:6].cpu().long(), new) and (out[:, :2] == -5).all() and (out[:, 6:] == -5).all()
    assert torch.equal(wide[:, 7:137].cpu(), want[0]) and (wide[:, :7] == 9).all() and (wide[:, 137:] == 9).all()
    same = ssu.reorder_states([], ts[:, :1].expand(3, 4), tp)  # one slot for all: no copies, the slot itself
    assert torch.equal(same.cpu(), ts[:, :1].expand(3, 4).cpu())


def test_large_slots_and_offsets():
    """Slots of 1.2 GB: offsets beyond 32 bits."""
    n = 1_200_000_003
    p = torch.zeros(4, n, dtype=torch.uint8, device="cuda")
    p[1, ::1000] = 7
    p[1, -1] = 11
    say("slots of %d bytes" % n)
    out = ssu.reorder_states(p, torch.tensor([[1, 3, 0]], device="cuda"), torch.tensor([[0, 0, 2]], device="cuda"))
    assert out.tolist() == [[1, 3, 0]]
    assert torch.equal(p[3], p[1]) and not p[0].any() and not p[2].any()


def test_streams_and_graph():
    pools, slots, parents = inputs(4, 6, [((3, 16, 32), torch.float32), ((64, 3), torch.bfloat16)], seed=8)
    say("streams and graph")
    d = [p.cuda() for p in pools]
    ds, dp = slots.int().cuda(), parents.int().cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = ssu.reorder_states(d, ds, dp)
    s.synchronize()
    want, new = S.reorder(pools, slots, parents)
    assert torch.equal(out.cpu().long(), new) and all(torch.equal(a.cpu(), b) for a, b in zip(d, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ssu.reorder_states(d, ds, dp)
    for i in range(4):
        pools, slots, parents = inputs(4, 6, [((3, 16, 32), torch.float32), ((64, 3), torch.bfloat16)], seed=30 + i, low=-1)
        for a, b in zip(d, pools):
            a.copy_(b)
        ds.copy_(slots)
        dp.copy_(parents)
        g.replay()
        torch.cuda.synchronize()
        want, new = S.reorder(pools, slots, parents)
        assert torch.equal(out.cpu().long(), new) and all(torch.equal(a.cpu(), b) for a, b in zip(d, want))
