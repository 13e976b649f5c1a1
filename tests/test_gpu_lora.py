"""add_lora against its definition in float64 (search_ref.lora, which says what it may be off by)."""
import math

import pytest
import torch

import layer_ref as R
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
    print("[gpu] add_lora", *a, flush=True)


def inputs(rows, k, n, rank, adapters, dt, seed=0, none=0.2, order="mixed"):
    g = torch.Generator().manual_seed(seed)
    c = {"y": torch.randn(rows, n, generator=g).to(DT[dt]), "x": (2 * torch.randn(rows, k, generator=g)).to(DT[dt]),
         "a": (torch.randn(adapters, rank, k, generator=g) / math.sqrt(k)).to(DT[dt]),
         "b": torch.randn(adapters, n, rank, generator=g).to(DT[dt]),
         "adapter": torch.randint(0, adapters, (rows,), generator=g).to(torch.int32),
         "scale": 0.5 + torch.rand(adapters, generator=g)}
    if order == "runs":
        c["adapter"] = torch.sort(c["adapter"]).values
    c["adapter"][torch.rand(rows, generator=g) < none] = -1
    return c


def run(c, scale=True, x=None):
    d = {k: v.cuda() for k, v in c.items()}
    say("x", tuple(c["x"].shape), c["x"].dtype, "n", c["y"].shape[1], "a", tuple(c["a"].shape))
    y = d["y"]
    r = ssu.add_lora(y, d["x"] if x is None else x, d["a"], d["b"], d["adapter"], d["scale"] if scale else None)
    torch.cuda.synchronize()
    assert r is y
    return y.cpu()


def check(y, c, scale=True, x=None):
    want, tol = S.lora(c["y"], c["x"] if x is None else x, c["a"], c["b"], c["adapter"], c["scale"] if scale else None)
    off = (y.double() - want).abs() - tol
    assert (off <= 0).all(), "%d of %d off, by up to %g" % ((off > 0).sum(), off.numel(), off.max())
    rest = (c["adapter"] < 0) | (c["adapter"] >= c["a"].shape[0])
    assert torch.equal(y[rest].view(torch.uint8), c["y"][rest].view(torch.uint8))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rank", [1, 3, 4, 8, 15, 16, 17, 20, 32, 33, 64, 65, 100, 127, 128])
def test_ranks(rank, dt):
    c = inputs(37, 200, 150, rank, 3, dt, seed=rank)
    check(run(c), c)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k", [1, 7, 8, 31, 32, 33, 255, 256, 257, 1024, 2592, 4100])
def test_inner_sizes(k, dt):
    c = inputs(19, k, 70, 16, 4, dt, seed=k)
    check(run(c), c)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 31, 33, 63, 64, 65, 255, 257, 513, 1111])
def test_outputs(n, dt):
    c = inputs(21, 96, n, 12, 4, dt, seed=n)
    check(run(c, scale=False), c, scale=False)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 127, 128, 129, 255, 256, 257, 511, 513, 2047, 2048, 2049, 5000])
@pytest.mark.parametrize("adapters", [1, 3, 50])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_rows_and_adapters(rows, adapters, order):
    c = inputs(rows, 160, 72, 8, adapters, "bf16", seed=rows + adapters, order=order)
    check(run(c), c)


@pytest.mark.parametrize("rows,adapters,order", [(8191, 3, "mixed"), (8193, 1, "runs"), (20000, 40, "mixed"), (20000, 4096, "mixed"), (30001, 9, "runs")])
def test_more_rows_than_the_lists_take_at_once(rows, adapters, order):
    c = inputs(rows, 64, 40, 4, adapters, "bf16", seed=rows + adapters, order=order)
    check(run(c), c)


@pytest.mark.parametrize("rows", [1, 4, 700, 3000])
def test_many_adapters(rows):
    c = inputs(rows, 64, 24, 4, 4096, "f16", seed=rows)
    check(run(c), c)


@pytest.mark.parametrize("rows,rank", [(60, 16), (60, 128), (250, 20), (250, 64), (2500, 16), (2500, 64), (2500, 128)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_large_inner_and_ranks(rows, rank, dt):
    c = inputs(rows, 2100, 130, rank, 5, dt, seed=rank, order="runs")
    check(run(c), c)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows,k,rank", [(1, 32, 4), (5, 4096, 16), (40, 544, 33), (300, 1024, 64), (2300, 288, 16), (2300, 288, 128)])
def test_codes(fmt, rows, k, rank):
    c = inputs(rows, k, 90, rank, 3, "bf16", seed=rows)
    x = torch.randn(rows, k, generator=torch.Generator().manual_seed(1)) * 3
    codes, scales = ssu.mx_quantize(x.cuda(), fmt)
    v = R.decode(codes, scales, fmt)
    check(run(c, x=(codes, scales)), c, x=v)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rank", [16, 32, 64, 128])
@pytest.mark.parametrize("k", [128, 512, 648, 4096, 4104])
def test_many_rows_in_whole_lines(dt, rank, k):
    """Rows that LDS-DMA can fetch: whole stages, an end that is none, several slices of k."""
    c = inputs(300, k, 136, rank, 3, dt, seed=k + rank)
    check(run(c), c)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("rank", [16, 32, 64, 128])
@pytest.mark.parametrize("k", [128, 640, 4096, 4192])
def test_many_rows_of_codes(fmt, rank, k):
    c = inputs(300, k, 70, rank, 3, "bf16", seed=k + rank)
    x = torch.randn(300, k, generator=torch.Generator().manual_seed(k)) * 3
    x[7, 40] = math.inf  # a block of NaNs, in a row that no adapter takes
    c["adapter"][7] = -1
    codes, scales = ssu.mx_quantize(x.cuda(), fmt)
    v = R.decode(codes, scales, fmt)
    check(run(c, x=(codes, scales)), c, x=v)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows", [40, 300])
def test_codes_off_any_alignment(fmt, rows):
    c = inputs(rows, 608, 70, 16, 3, "bf16", seed=rows)
    x = torch.randn(rows, 608, generator=torch.Generator().manual_seed(2))
    codes, scales = ssu.mx_quantize(x.cuda(), fmt)
    v = R.decode(codes, scales, fmt)
    wide = torch.full((rows, codes.shape[1] + 13), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, 3:3 + codes.shape[1]] = codes
    wide_scales = torch.full((rows, 27), 255, dtype=torch.uint8, device="cuda")
    wide_scales[:, 5:24] = scales
    check(run(c, x=(wide[:, 3:3 + codes.shape[1]], wide_scales[:, 5:24])), c, x=v)


@pytest.mark.parametrize("rows", [200, 1500])
def test_few_of_many_adapters(rows):
    """Most rows of one adapter, most adapters without a row, and rows before the matrix that LDS-DMA cannot fetch whole."""
    c = inputs(rows, 256, 300, 16, 64, "bf16", seed=rows, none=0.05)
    c["adapter"][c["adapter"] >= 0] = 37
    c["adapter"][::50] = 3
    check(run(c), c)
    wide = torch.zeros(rows, 259, dtype=torch.bfloat16)
    wide[:, 1:257] = c["x"]
    d = {k: v.cuda() for k, v in c.items()}
    y = ssu.add_lora(d["y"], wide.cuda()[:, 1:257], d["a"], d["b"], d["adapter"], d["scale"])
    check(y.cpu(), c)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_codes_that_are_not_finite(fmt):
    """A block of NaNs, and the smallest and largest scales."""
    c = inputs(6, 64, 40, 8, 2, "bf16", none=0.0)
    x = torch.randn(6, 64)
    x[1, 40] = math.nan
    codes, scales = ssu.mx_quantize(x.cuda(), fmt)
    scales[2] = 0    # 2^-127
    scales[3] = 1
    scales[4] = 200
    v = R.decode(codes, scales, fmt)
    y = run(c, x=(codes, scales))
    assert torch.isnan(y[1]).all()
    keep = [0, 2, 3, 5]
    check(y[keep], {**c, "y": c["y"][keep], "adapter": c["adapter"][keep]}, x=v[keep])
    want, tol = S.lora(c["y"], v, c["a"], c["b"], c["adapter"], c["scale"])
    assert ((y[4].double() - want[4]).abs() <= tol[4]).all()


def test_adapters_do_not_meet():
    """NaN and infinity in one adapter, or in one row, stay with their rows."""
    for rows in (50, 2600):
        c = inputs(rows, 100, 80, 16, 4, "bf16", seed=rows, none=0.1)
        c["a"][1, 3, 5] = math.nan
        c["b"][2, 7, 2] = math.inf
        c["x"][10] = math.nan
        c["scale"][3] = math.nan
        c["adapter"][10], c["adapter"][11] = 0, 0
        y = run(c)
        mine = c["adapter"] == 0
        mine[10] = False
        mine |= c["adapter"] == -1
        check(y[mine], {**c, "y": c["y"][mine], "x": c["x"][mine], "adapter": c["adapter"][mine]})
        assert torch.isnan(y[10]).all() and torch.isnan(y[c["adapter"] == 1]).all() and torch.isnan(y[c["adapter"] == 3]).all()
        two = c["adapter"] == 2
        assert not torch.isfinite(y[two][:, 7]).any()
        others = [i for i in range(80) if i != 7]
        check(y[two][:, others], {**c, "y": c["y"][two][:, others], "x": c["x"][two], "adapter": c["adapter"][two],
                                  "b": c["b"][:, others]})


def test_large_values_in_f16():
    """h beyond f16's range, and far below it: y has room for the result."""
    c = inputs(30, 64, 50, 8, 3, "f16", none=0.0)
    c["x"] = (c["x"].float() * 2000).half()
    c["a"] = (c["a"].float() * 300).half()
    c["b"] = (c["b"].float() * 2.0 ** -16).half()
    c["scale"] = torch.tensor([1.0, 2.0 ** -6, 2.0 ** -30])
    check(run(c), c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_dimensions(dt):
    c = inputs(12, 75, 61, 10, 3, dt, seed=2)
    want = run(c)
    check(want, c)
    d = {k: v.cuda() for k, v in c.items()}
    y = torch.full((12, 91), 5.0, dtype=DT[dt], device="cuda")
    y[:, 11:72] = d["y"]
    x = torch.full((12, 103), math.nan, dtype=DT[dt], device="cuda")
    x[:, 1:76] = d["x"]
    a = torch.full((3, 13, 90), math.nan, dtype=DT[dt], device="cuda")
    a[:, 1:11, 3:78] = d["a"]
    b = torch.full((61, 3, 17), math.nan, dtype=DT[dt], device="cuda")
    b[:, :, 5:15] = d["b"].transpose(0, 1)
    ids = torch.full((24,), 2, dtype=torch.int64, device="cuda")[::2]
    ids.copy_(d["adapter"])
    scale = torch.full((9,), math.nan, device="cuda")[::3]
    scale.copy_(d["scale"])
    ssu.add_lora(y[:, 11:72], x[:, 1:76], a[:, 1:11, 3:78], b[:, :, 5:15].transpose(0, 1), ids, scale)
    assert torch.equal(y[:, 11:72].cpu(), want) and (y[:, :11] == 5).all() and (y[:, 72:] == 5).all()
    y3 = d["y"].clone().view(3, 4, 61)
    ssu.add_lora(y3, d["x"].view(3, 4, 75), d["a"], d["b"], d["adapter"], d["scale"])
    assert torch.equal(y3.view(12, 61).cpu(), want)
    one = d["y"][0].clone()
    ssu.add_lora(one, d["x"][0], d["a"], d["b"], d["adapter"][:1], d["scale"])
    assert torch.equal(one.cpu(), want[0])
    # one adapter's weights under several numbers
    y4 = d["y"].clone()
    ssu.add_lora(y4, d["x"], d["a"][:1].expand(7, 10, 75), d["b"][:1].expand(7, 61, 10), d["adapter"], None)
    c2 = {**c, "a": c["a"][:1].expand(7, 10, 75), "b": c["b"][:1].expand(7, 61, 10)}
    check(y4.cpu(), c2, scale=False)


def test_numbers_out_of_range():
    c = inputs(40, 48, 56, 8, 3, "bf16")
    c["adapter"] = torch.tensor([0, 1, 2, 3, -1, -2 ** 31, 2 ** 31 - 1, 1] * 5, dtype=torch.int32)
    want = run(c)
    check(want, c)
    c["adapter"] = c["adapter"].long()
    c["adapter"][3] = 2 ** 32  # 0 in its low half
    c["adapter"][4] = -2 ** 33
    assert torch.equal(run(c), want)


@pytest.mark.parametrize("rows", [90, 2200])
def test_repeats_streams_and_graph(rows):
    c = inputs(rows, 1200, 140, 16, 6, "bf16", seed=rows)
    want = run(c)
    for _ in range(3):
        assert torch.equal(run(c), want)
    d = {k: v.cuda() for k, v in c.items()}
    y = d["y"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ssu.add_lora(y, d["x"], d["a"], d["b"], d["adapter"], d["scale"])
    s.synchronize()
    assert torch.equal(y.cpu(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssu.add_lora(y, d["x"], d["a"], d["b"], d["adapter"], d["scale"])
    for i in range(4):
        new = inputs(rows, 1200, 140, 16, 6, "bf16", seed=50 + i)
        for name in ("x", "adapter"):
            d[name].copy_(new[name])
        y.copy_(new["y"])
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.copy_(new["y"])
        assert torch.equal(got, ssu.add_lora(y, d["x"], d["a"], d["b"], d["adapter"], d["scale"]))


def test_offsets_beyond_32_bits():
    c = inputs(3, 64, 72, 8, 2, "bf16", none=0.0)
    stride = 1_200_000_008
    d = {k: v.cuda() for k, v in c.items()}
    big = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device="cuda")
    y = big.as_strided((3, 72), (stride, 1), 0)
    x = big.as_strided((3, 64), (stride, 1), 100)
    y.copy_(d["y"])
    x.copy_(d["x"])
    say("rows %d elements apart" % stride)
    ssu.add_lora(y, x, d["a"], d["b"], d["adapter"], d["scale"])
    check(y.cpu(), c)


def test_empty():
    def z(*shape, dt=torch.bfloat16):
        return torch.ones(shape, dtype=dt, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for y, x, a, b in ((z(0, 8), z(0, 16), z(2, 4, 16), z(2, 8, 4)), (z(4, 8), z(4, 0), z(2, 4, 0), z(2, 8, 4)),
                       (z(4, 8), z(4, 16), z(0, 4, 16), z(0, 8, 4)), (z(4, 8), z(4, 16), z(2, 0, 16), z(2, 8, 0)),
                       (z(4, 0), z(4, 16), z(2, 4, 16), z(2, 0, 4))):
        r = ssu.add_lora(y, x, a, b, ids[:y.shape[0]])
        assert r is y and (y == 1).all()
