"""mx_quantize and mx_linear against their definitions (layer_ref).

Quantisation is exact: bytes are compared. Products: E2M1 x E2M1 times powers of two
are multiples of a power of two, so with scales of a narrow range every partial sum
is a whole number of 2^-2 below 2^22 and the fp32 result is exact. In general the
sum of k products in fp32 is off by at most (k / 64 + 64) 2^-24 of the sum of their
magnitudes for MXFP4; the E4M3 products of one instruction keep about 13 bits below
the largest (measured: 1.2e-4 of the sum of magnitudes at the worst of random
codes over the whole range), 2^-12 of it here; then the output's rounding."""
import pytest
import torch

import layer_ref as R
import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------- quantisation

def check_codes(x, fmt, codes, scales):
    q, byte = R.quantize(x, fmt)
    assert torch.equal(scales.cpu(), byte)
    bad = byte == 255
    values = R.decode(codes.cpu(), torch.full_like(byte, 127), fmt)
    want = torch.where(bad.repeat_interleave(32, -1), torch.zeros_like(q), q)
    assert torch.equal(values, want)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (5, 96), (257, 2592), (2, 8192), (1000, 32)])
def test_quantize(fmt, dt, rows, k):
    g = torch.Generator().manual_seed(rows + k)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, k // 32), generator=g).float()).repeat_interleave(32, 1)
    x = x.to(DT[dt])
    say("[gpu] mx_quantize", fmt, dt, rows, k)
    check_codes(x, fmt, *ssu.mx_quantize(x.cuda(), fmt))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_quantize_special_values(fmt):
    step = {"mxfp8": 1 / 16, "mxfp4": 0.25}[fmt]
    x = (torch.arange(-64, 64).float() * step).reshape(4, 32)        # every tie of the lower binades
    x[:, 0] = 1.75 * 2.0 ** R.EMAX[fmt]
    rows = [x, torch.zeros(1, 32), torch.full((1, 32), 1e-41), torch.full((1, 32), 3e38), -torch.full((1, 32), 2.0 ** -126)]
    for v in (float("inf"), -float("inf"), float("nan")):
        r = torch.ones(1, 32)
        r[0, 31] = v
        rows.append(r)
    x = torch.cat(rows)
    codes, scales = ssu.mx_quantize(x.cuda(), fmt)
    check_codes(x, fmt, codes, scales)
    assert (scales[-3:] == 255).all() and torch.isnan(R.decode(codes, scales, fmt)[-3:]).all()


def test_quantize_strided_rows():
    x = torch.randn(9, 200, dtype=torch.float32).to(torch.bfloat16)
    d = x.cuda()[:, 3:163]
    for fmt in ("mxfp8", "mxfp4"):
        check_codes(x[:, 3:163], fmt, *ssu.mx_quantize(d, fmt))
    codes, scales = ssu.mx_quantize(x.cuda()[:, :160].reshape(3, 3, 160))
    assert codes.shape == (3, 3, 80) and scales.shape == (3, 3, 5)


# ---------------------------------------------------------------- products

def weights(n, k, g, lo=125, hi=129):
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(lo, hi + 1, (n, k // 32), generator=g, dtype=torch.uint8)
    return codes, scales


def acts(m, k, fmt, g, lo=126, hi=128):
    scales = torch.randint(lo, hi + 1, (m, k // 32), generator=g, dtype=torch.uint8)
    if fmt == "mxfp4":
        return torch.randint(0, 256, (m, k // 2), generator=g, dtype=torch.uint8), scales
    # 0, +-1, +-2, +-4: products whose alignment loses nothing
    v = torch.tensor([0.0, 1.0, 2.0, 4.0, -1.0, -2.0, -4.0])[torch.randint(0, 7, (m, k), generator=g)]
    return v.to(torch.float8_e4m3fn).view(torch.uint8), scales


SHAPES = [(1, 1, 32), (1, 33, 64), (2, 64, 96), (1, 4096, 512), (3, 100, 160), (16, 128, 1024), (17, 48, 2592), (31, 130, 288),
          (32, 32, 64), (33, 257, 128), (64, 512, 4096), (65, 300, 544), (100, 1000, 992), (129, 129, 1056), (128, 256, 512),
          (255, 511, 256), (256, 256, 2048), (300, 770, 352), (513, 640, 640), (1, 18560, 64), (700, 72, 8192), (2050, 1030, 96)]


# enough rows and outputs for the larger tiles
LARGE = [(2100, 2090, 160), (1100, 2080, 1312), (4200, 4130, 288), (5000, 5000, 544)]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m,n,k", SHAPES + LARGE)
def test_exact_products(m, n, k, fmt):
    """Sums that fp32 holds exactly, in every output type and with a bias."""
    g = torch.Generator().manual_seed(m * 7 + n * 3 + k)
    a, sa = acts(m, k, fmt, g)
    w, sw = weights(n, k, g)
    bias = torch.randint(-8, 9, (n,), generator=g).float()
    ref = (R.decode(a, sa, fmt).cuda() @ R.decode(w, sw, "mxfp4").cuda().t()).cpu() + bias.double()
    say("[gpu] mx_linear", fmt, m, n, k)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        y = ssu.mx_linear((a.cuda(), sa.cuda()), w.cuda(), sw.cuda(), bias=bias.cuda(), out_dtype=dt)
        assert torch.equal(y.cpu(), ref.float().to(dt)), dt


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (1, 1030, 4096), (4, 256, 2592), (8, 512, 8192), (40, 96, 1024), (300, 520, 2080), (1025, 260, 512)])
def test_float_activations(m, n, k, dt, fmt):
    g = torch.Generator().manual_seed(m + n + k)
    x = (torch.randn(m, k, generator=g) * torch.where(torch.rand(k, generator=g) < 0.02, 10.0, 1.0)).to(DT[dt])
    w, sw = ssu.mx_quantize((torch.randn(n, k, generator=g) / k ** 0.5).cuda())
    say("[gpu] mx_linear of floats", fmt, dt, m, n, k)
    y = ssu.mx_linear(x.cuda(), w, sw, activation=fmt)
    q, byte = R.quantize(x, fmt)
    a = q * torch.ldexp(torch.ones(byte.shape, dtype=torch.float64), byte.int() - 127).repeat_interleave(32, -1)
    wd = R.decode(w, sw, "mxfp4")
    ref = (a.cuda() @ wd.cuda().t()).cpu()
    mag = (a.abs().cuda() @ wd.abs().cuda().t()).cpu()
    rel = (k / 64 + 64) * 2.0 ** -24 + (2.0 ** -12 if fmt == "mxfp8" else 0)
    tol = rel * mag + R.ROUND[DT[dt]] * ref.abs() + R.TINY[DT[dt]]
    assert y.dtype == DT[dt] and ((y.cpu().double() - ref).abs() <= tol).all()
    # the same from codes made beforehand
    pair = ssu.mx_linear(ssu.mx_quantize(x.cuda(), fmt), w, sw, out_dtype=DT[dt])
    assert torch.equal(pair, y)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m", [1, 20, 300])
def test_whole_scale_range(m, fmt):
    """Scale bytes from 0 to 254 where the sums stay in range: one row each."""
    k, n = 256, 96
    g = torch.Generator().manual_seed(m)
    a, sa = acts(m, k, fmt, g, 127, 127)
    w, sw = weights(n, k, g, 127, 127)
    s = torch.randint(0, 255, (n, 1), generator=g)
    s[0], s[1] = 0, 254
    sw = s.expand(n, k // 32).to(torch.uint8).contiguous()
    sa[:] = 100
    ref = (R.decode(a, sa, fmt) @ R.decode(w, sw, "mxfp4").t())
    y = ssu.mx_linear((a.cuda(), sa.cuda()), w.cuda(), sw.cuda(), out_dtype=torch.float32).cpu()
    fits = ref.abs() >= 2.0 ** -126
    assert torch.equal(y[fits], ref.float()[fits])
    assert ((y.double() - ref).abs()[~fits] <= 2.0 ** -126).all()


@pytest.mark.parametrize("m", [1, 5, 40, 300])
def test_not_finite_rows(m):
    """An infinity or a NaN in a row of activations makes that row NaN and no other;
    so does a NaN scale in a row of weights for its column."""
    k, n = 320, 140
    g = torch.Generator().manual_seed(m)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16)
    x[m // 2, k - 1] = float("inf")
    x[0, 3] = float("nan")
    w, sw = ssu.mx_quantize(torch.randn(n, k, generator=g).cuda())
    sw[n - 1, 4] = 255
    for fmt in ("mxfp8", "mxfp4"):
        y = ssu.mx_linear(x.cuda(), w, sw, activation=fmt).cpu()
        want = torch.zeros(m, n, dtype=torch.bool)
        want[m // 2] = want[0] = True
        want[:, n - 1] = True
        assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("m", [1, 7, 150])
def test_strides(m):
    """Row slices of wider tensors, for every operand, and an output between guards."""
    k, n = 288, 200
    g = torch.Generator().manual_seed(m)
    for fmt in ("mxfp8", "mxfp4"):
        a, sa = acts(m, k, fmt, g)
        w, sw = weights(n, k, g)
        ref = R.decode(a, sa, fmt) @ R.decode(w, sw, "mxfp4").t()

        def wide(t, before, after):
            big = torch.full((t.shape[0], before + t.shape[1] + after), 255, dtype=torch.uint8, device="cuda")
            big[:, before:before + t.shape[1]] = t.cuda()
            return big[:, before:before + t.shape[1]]
        out = torch.full((m, n + 9), 5.0, dtype=torch.float32, device="cuda")
        y = ssu.mx_linear((wide(a, 16, 32 + -a.shape[1] % 16), wide(sa, 3, 2)), wide(w, 32, 48 + -w.shape[1] % 16), wide(sw, 1, 6),
                          out=out[:, 3:n + 3])
        assert torch.equal(y.cpu(), ref.float())
        assert (out[:, :3] == 5).all() and (out[:, n + 3:] == 5).all()


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(4347, 4001, 96), (4001, 4347, 608), (4354, 3841, 64)])
def test_last_round_of_tiles(m, n, k, fmt):
    """A few tiles more than whole rounds of them, below and on the right: float activations that
    are codes again, a bias in the outputs' type, strided outputs between guards."""
    g = torch.Generator().manual_seed(m + n + k)
    a, sa = acts(m, k, fmt, g)
    x = R.decode(a, sa, fmt).float()
    w, sw = weights(n, k, g)
    bias = torch.randint(-8, 9, (n,), generator=g).float()
    ref = R.decode(a, sa, fmt).cuda() @ R.decode(w, sw, "mxfp4").cuda().t() + bias.double().cuda()
    say("[gpu] mx_linear, last round", fmt, m, n, k)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((m, n + 5), 5.0, dtype=dt, device="cuda")
        ssu.mx_linear(x.cuda(), w.cuda(), sw.cuda(), bias=bias.cuda().to(dt), activation=fmt, out=out[:, 2:n + 2])
        assert torch.equal(out[:, 2:n + 2], ref.float().to(dt)), dt
        assert (out[:, :2] == 5).all() and (out[:, n + 2:] == 5).all()


def test_leading_dimensions_and_empty():
    g = torch.Generator().manual_seed(0)
    w, sw = (t.cuda() for t in weights(64, 128, g))
    x = torch.randn(2, 3, 128, generator=g).to(torch.bfloat16).cuda()
    y = ssu.mx_linear(x, w, sw)
    assert y.shape == (2, 3, 64) and torch.equal(y.view(6, 64), ssu.mx_linear(x.view(6, 128), w, sw))
    assert torch.equal(ssu.mx_linear(x[0, 0], w, sw), y[0, 0])
    assert ssu.mx_linear(x[:0], w, sw).shape == (0, 3, 64)
    # no inner size: the bias alone
    b = torch.arange(5, dtype=torch.float32, device="cuda")
    z = ssu.mx_linear(torch.empty(2, 0, dtype=torch.float32, device="cuda"), torch.empty(5, 0, dtype=torch.uint8, device="cuda"),
                      torch.empty(5, 0, dtype=torch.uint8, device="cuda"), bias=b)
    assert torch.equal(z, b.expand(2, 5))


def test_offsets_beyond_32_bits():
    """Weight and output rows that lie more than 2^32 bytes apart."""
    g = torch.Generator().manual_seed(4)
    k, n, m = 64, 3, 3
    a, sa = acts(m, k, "mxfp8", g)
    w, sw = weights(n, k, g)
    ref = R.decode(a, sa, "mxfp8") @ R.decode(w, sw, "mxfp4").t()
    stride = 2_400_000_016
    big = torch.empty(2 * stride + 64, dtype=torch.uint8, device="cuda")
    wv = big.as_strided((n, k // 2), (stride, 1))
    wv.copy_(w.cuda())
    say("[gpu] mx_linear, weight rows %d bytes apart" % stride)
    y = ssu.mx_linear((a.cuda(), sa.cuda()), wv, sw.cuda(), out_dtype=torch.float32)
    assert torch.equal(y.cpu(), ref.float())
    av = big.as_strided((m, k), (stride, 1))
    av.copy_(a.cuda())
    out = torch.empty(2 * (stride // 2) + 8, dtype=torch.float32, device="cuda").as_strided((m, n), (stride // 2, 1))
    y = ssu.mx_linear((av, sa.cuda()), w.cuda(), sw.cuda(), out=out)
    assert torch.equal(y.cpu(), ref.float())


def test_streams_and_graph():
    g = torch.Generator().manual_seed(2)
    for m in (1, 40):
        x = torch.randn(m, 1024, generator=g).to(torch.bfloat16).cuda()
        w, sw = ssu.mx_quantize(torch.randn(520, 1024, generator=g).cuda())
        want = ssu.mx_linear(x, w, sw)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = []
        for s in streams:  # calls that overlap, each with its own stream's workspace
            with torch.cuda.stream(s):
                got.append([ssu.mx_linear(x, w, sw) for _ in range(4)])
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for ys in got for y in ys)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ssu.mx_linear(x, w, sw)
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                y = ssu.mx_linear(x, w, sw)
        for i in range(4):
            x.copy_(torch.randn(m, 1024, generator=g).to(torch.bfloat16).cuda())
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, ssu.mx_linear(x, w, sw))
