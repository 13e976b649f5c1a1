"""add_rms_norm against its definition in float64 (layer_ref.norm).

Tolerance of a result in x's dtype: one rounding to it (half an ulp, ROUND), and
1e-5 of the magnitudes that the fp32 steps work on: the sum of squares (a
tree over a few hundred terms a lane: below 64 * 2^-24), the reciprocal square
root, and the gate's exponential, whose error grows as |z| 2^-23 (|z| < 40 here).
An MX result: the distance of a code from the value it stands for is at most
half the step there, plus the same 1e-5 (a scale may differ where that moves a
block's largest magnitude over a power of two)."""
import numpy as np
import pytest
import torch

import layer_ref as R
import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
REL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def say(*a):
    print(*a, flush=True)


def inputs(rows, dim, dt, seed=0, residual=None, gate=False, weight=None):
    g = torch.Generator().manual_seed(seed)
    c = {"x": (torch.randn(rows, dim, generator=g) * 3).to(DT[dt])}
    c["weight"] = (1 + 0.3 * torch.randn(dim, generator=g)).to(DT[weight or dt])
    c["residual"] = (torch.randn(rows, dim, generator=g) * 5).to(DT[residual]) if residual else None
    c["gate"] = (torch.randn(rows, dim, generator=g) * 4).to(DT[dt]) if gate else None
    return c


def dev(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def check_same(y, ref, size, dt):
    y, tol = y.cpu().double(), R.ROUND[dt] * ref.abs() + R.TINY[dt] + REL * size
    bad = (y - ref).abs() > tol
    assert not bad.any(), "%d of %d off, by up to %g" % (bad.sum(), bad.numel(), ((y - ref).abs() - tol).max())


def check_mx(codes, scales, ref, size, fmt):
    rows = ref.shape[0]
    blocks = ref.reshape(rows, -1, 32)
    amax = blocks.abs().amax(-1)
    want = R.quantize(ref, fmt)[1]
    got = scales.cpu().reshape(want.shape)
    frac, _ = torch.frexp(amax)
    slack = 2 * REL * (size.reshape(blocks.shape).amax(-1) / amax.clamp(min=1e-300))
    near = ((frac - 0.5).abs() < slack) | ((1 - frac) < slack) | (amax == 0)
    assert ((got == want) | near).all()
    v = torch.ldexp(blocks, -(got.int() - 127)[..., None]).reshape(rows, -1)
    code = R.decode(codes.cpu().reshape(rows, -1), torch.full_like(got, 127), fmt)
    top = R.LARGEST[fmt]
    err = (code - v.clamp(-top, top)).abs()
    off = torch.ldexp(size.reshape(blocks.shape), -(got.int() - 127)[..., None]).reshape(rows, -1) * REL
    assert (err <= R.step(v, fmt) / 2 + off).all(), float((err - R.step(v, fmt) / 2 - off).max())


def run(c, **kw):
    say("[gpu] norm", tuple(c["x"].shape), c["x"].dtype, {k: v for k, v in kw.items() if k != "eps"})
    d = dev(c)
    r = ssu.add_rms_norm(d["x"], d["weight"], residual=d["residual"], gate=d["gate"], **kw)
    torch.cuda.synchronize()
    return r


DIMS = [1, 2, 7, 8, 31, 33, 64, 100, 255, 257, 512, 1000, 1023, 2048, 2561, 4096, 4097, 8192, 8200, 16384, 16385, 40000]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_widths(dim, dt):
    c = inputs(3, dim, dt, seed=dim, residual=dt)
    y, r = run(c)
    ref, u, size = R.norm(c["x"], c["weight"], c["residual"])
    check_same(y, ref, size, DT[dt])
    assert torch.equal(r.cpu(), u.float().to(DT[dt]))  # one exact sum of two such numbers, rounded


@pytest.mark.parametrize("rows", [1, 2, 5, 63, 300, 1500])
def test_row_counts(rows):
    c = inputs(rows, 768, "bf16", seed=rows)
    y = run(c)
    ref, _, size = R.norm(c["x"], c["weight"])
    check_same(y, ref, size, DT["bf16"])


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gate,residual", [(False, None), (True, None), (False, "same"), (True, "f32")])
@pytest.mark.parametrize("dim,groups", [(64, 1), (96, 3), (1024, 1), (2048, 8), (4096, 1), (8192, 8), (8224, 1), (20480, 2)])
def test_forms(fmt, dt, gate, residual, dim, groups):
    c = inputs(4, dim, dt, seed=dim + groups, residual=dt if residual == "same" else residual, gate=gate,
               weight="f32" if gate else None)
    r = run(c, groups=groups, eps=1e-3, out_format=fmt)
    ref, u, size = R.norm(c["x"], c["weight"], c["residual"], c["gate"], groups, 1e-3)
    if residual:
        r, res = r
        rt = c["residual"].dtype
        mag = c["residual"].double().abs() + (u - c["residual"].double()).abs()
        err = (res.cpu().double() - u).abs()
        assert (err <= R.ROUND[rt] * u.abs() + R.TINY[rt] + REL * mag * (1 if gate else 0) + 2.0 ** -24 * mag).all()
    if fmt is None:
        check_same(r, ref, size, DT[dt])
    else:
        check_mx(*r, ref, size, fmt)


@pytest.mark.parametrize("fmt", [None, "mxfp8"])
def test_strides_alignment_and_leading_dimensions(fmt):
    c = inputs(12, 96, "f16", seed=3, residual="f16", gate=True)
    ref, u, size = R.norm(c["x"], c["weight"], c["residual"], c["gate"])
    wide = {k: torch.full((12, 131), 9.0, dtype=torch.float16, device="cuda") for k in ("x", "residual", "gate")}
    for i, k in enumerate(wide):  # rows at odd element offsets and an odd stride
        wide[k][:, 2 * i + 1:2 * i + 97] = c[k].cuda()
        wide[k] = wide[k][:, 2 * i + 1:2 * i + 97]
    out = None if fmt else torch.full((12, 103), 7.0, dtype=torch.float16, device="cuda")
    say("[gpu] norm strided", fmt)
    r, res = ssu.add_rms_norm(wide["x"], c["weight"].cuda(), wide["residual"], wide["gate"], out_format=fmt,
                              out=None if fmt else out[:, 5:101], residual_out=wide["residual"])
    torch.cuda.synchronize()
    assert res.data_ptr() == wide["residual"].data_ptr()  # in place
    if fmt:
        check_mx(*r, ref, size, fmt)
    else:
        check_same(r, ref, size, torch.float16)
        assert (out[:, :5] == 7).all() and (out[:, 101:] == 7).all()
    d = dev(c)
    r3, res3 = ssu.add_rms_norm(d["x"].view(3, 4, 96), d["weight"], d["residual"].view(3, 4, 96),
                                d["gate"].view(3, 4, 96), out_format=fmt)
    assert res3.shape == (3, 4, 96)
    a, b = (r, r3) if fmt is None else (r[0], r3[0])
    assert torch.equal(b.reshape(a.shape), a)
    # the output over the input
    x = d["x"].clone()
    if fmt is None:
        y, _ = ssu.add_rms_norm(x, d["weight"], d["residual"], d["gate"], out=x)
        assert y is x and torch.equal(x, r)


def test_broadcast_rows():
    c = inputs(1, 512, "bf16", seed=5, residual="bf16")
    many = c["x"].cuda().expand(7, 512)
    y, r = ssu.add_rms_norm(many, c["weight"].cuda(), c["residual"].cuda().expand(7, 512))
    one, r1 = run(c)
    assert torch.equal(y, one.expand(7, 512)) and torch.equal(r, r1.expand(7, 512))


@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
def test_special_values(fmt):
    x = torch.randn(6, 64, generator=torch.Generator().manual_seed(1))
    x[0] = 0            # y = 0 whatever eps
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] *= 1e18        # squares up to 1e36: still finite
    x[4] *= 1e-22       # squares below the smallest normal
    w = torch.ones(64)
    say("[gpu] norm special values", fmt)
    r = ssu.add_rms_norm(x.cuda(), w.cuda(), eps=1e-12, out_format=fmt)
    torch.cuda.synchronize()
    if fmt:
        codes, scales = r[0].cpu(), r[1].cpu()
        y = R.decode(codes, scales, fmt)
        assert torch.isnan(y[1]).all() and (scales[1] == 255).all()
        assert (scales[0] == 1).all() and (codes[0] == 0).all()
        keep = [0, 3, 4, 5]
        ref, _, size = R.norm(x[keep], w, eps=1e-12)
        check_mx(codes[keep], scales[keep], ref, size, fmt)
        # inf * 0 is a NaN, the rest of an infinite row is 0 (its other block finite)
        assert scales[2, 0] == 255 and torch.isnan(y[2, :32]).all() and (y[2, 32:] == 0).all()
    else:
        y = r.cpu()
        assert torch.isnan(y[1]).all()
        assert torch.isnan(y[2, 7]) and (y[2, :7] == 0).all() and (y[2, 8:] == 0).all()
        assert (y[0] == 0).all()
        ref, _, size = R.norm(x[3:], w, eps=1e-12)
        check_same(y[3:], ref, size, torch.float32)


def test_gate_extremes():
    """silu at large |z|: z for z >> 0, 0 for z << 0, and no NaN between."""
    z = torch.tensor([-1e4, -200.0, -90.0, -88.5, -50.0, 0.0, 50.0, 90.0, 200.0, 1e4]).repeat(1, 4)
    x = torch.ones_like(z)
    w = torch.ones(z.shape[1])
    res = torch.zeros_like(z)
    _, u = ssu.add_rms_norm(x.cuda(), w.cuda(), res.cuda(), z.cuda())
    want = z.double() * torch.sigmoid(z.double())
    assert ((u.cpu().double() - want).abs() <= 4e-6 * want.abs() + 1e-30).all(), (u.cpu(), want)


def test_offsets_beyond_32_bits():
    """Three rows 1.2e9 elements apart."""
    stride = 1_200_000_007
    c = inputs(3, 100, "bf16", seed=9)
    big = torch.empty(2 * stride + 128, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((3, 100), (stride, 1), 3)
    x.copy_(c["x"].cuda())
    say("[gpu] norm, rows %d elements apart" % stride)
    y = ssu.add_rms_norm(x, c["weight"].cuda(), out=x)
    ref, _, size = R.norm(c["x"], c["weight"])
    check_same(y, ref, size, torch.bfloat16)


def test_streams_and_graph():
    c = inputs(64, 4096, "bf16", seed=11, residual="bf16")
    d = dev(c)
    want, wres = run(c, out_format="mxfp8")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, res = ssu.add_rms_norm(d["x"], d["weight"], d["residual"], out_format="mxfp8")
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(res, wres)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, res = ssu.add_rms_norm(d["x"], d["weight"], d["residual"], out_format="mxfp8")
    for i in range(4):
        d["x"].copy_(c["x"].cuda() * (i + 1))
        g.replay()
        torch.cuda.synchronize()
        eager, er = ssu.add_rms_norm(d["x"], d["weight"], d["residual"], out_format="mxfp8")
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1]) and torch.equal(res, er)


def test_numpy_free_of_rows():
    """No rows: nothing launched, outputs of the right shape."""
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y = ssu.add_rms_norm(x, torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    assert y.shape == (0, 64) and np.prod(y.shape) == 0
