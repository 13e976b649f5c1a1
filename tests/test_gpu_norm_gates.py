"""Gates at the ends of their range: silu(z) = z sigmoid(z) is z, 0 and, at -inf, -inf times 0."""
import math

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


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", [None, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dim", [64, 4096, 40000])
def test_infinite_gates(dt, fmt, dim):
    """-inf makes its row NaN (u is one), +inf an infinite u there, as the definition does."""
    g = torch.Generator().manual_seed(dim)
    x = (1 + torch.rand(4, dim, generator=g)).to(DT[dt])
    z = torch.randn(4, dim, generator=g).to(DT[dt])
    z[1, 5], z[2, dim - 1] = -math.inf, math.inf
    res = torch.zeros(4, dim, dtype=torch.float32)
    w = torch.ones(dim, dtype=DT[dt])
    print("[gpu] infinite gates", dt, fmt, dim, flush=True)
    r, u = ssu.add_rms_norm(x.cuda(), w.cuda(), res.cuda(), z.cuda(), out_format=fmt)
    y = r.cpu() if fmt is None else R.decode(r[0].cpu(), r[1].cpu(), fmt)
    want, wu, _ = R.norm(x, w, res, z)
    assert torch.equal(torch.isnan(u.cpu()), torch.isnan(wu)) and torch.isnan(wu).sum() == 1
    assert torch.equal(torch.isinf(u.cpu()), torch.isinf(wu)) and torch.isinf(wu).sum() == 1
    assert torch.isnan(y[1]).all()
    if fmt is None:
        assert torch.equal(torch.isnan(y), torch.isnan(want))
    else:  # an infinite u: its block of y holds a NaN, the others are 0
        assert torch.isnan(y[2, -32:]).all() and (y[2, :-32] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_far_negative_gates(dt):
    """silu(z) down to where float32 ends: within 2^-21 of itself (the exponential and three products) and half
    of the smallest float32, 2^-150, times x; from -104 on it is 0 however large x is."""
    z = torch.tensor([-80.0, -86.5, -87.0, -87.5, -88.0, -89.0, -92.0, -95.0, -100.0, -103.0, -104.5, -120.0, -1e3, -1e4, -1e20, -3e38])
    z = z.repeat(8).to(DT[dt])[None]
    x = torch.full_like(z, 1e30)
    x[0, :32] = 3e37
    res = torch.zeros(z.shape)
    print("[gpu] far negative gates", dt, flush=True)
    for dim in (128, 16):  # both ways a gate is read: in registers, and one wave for a short part
        v, w = z[:, :dim], torch.ones(dim, dtype=DT[dt]).cuda()
        _, u = ssu.add_rms_norm(x[:, :dim].cuda(), w, res[:, :dim].contiguous().cuda(), v.cuda())
        want = x[:, :dim].double() * v.double() * torch.exp(v.double())
        err = (u.cpu().double() - want).abs()
        assert (err <= 2.0 ** -21 * want.abs() + 2.0 ** -150 * x[:, :dim].double()).all(), err
        assert (u.cpu()[v < -110] == 0).all()
