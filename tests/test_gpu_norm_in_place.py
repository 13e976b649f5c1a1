"""add_rms_norm over its own inputs (out is x, residual_out is residual) gives what it gives in other memory, bit for
bit: at parts whose last eight elements overlap the run before them, which two lanes or waves then
store, at parts that are read twice, and at the widths around both."""
import pytest
import torch

import mamba_selective_state_amd as ssu

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


@pytest.mark.parametrize("dim,groups", [(5, 1), (9, 1), (15, 1), (18, 2), (100, 1), (129, 1), (513, 1), (1025, 1), (2049, 1), (2561, 1), (4097, 1),
                                        (8191, 1), (16383, 1), (16386, 2), (20001, 1), (32767, 1), (32769, 1), (40001, 1), (120003, 3)])
@pytest.mark.parametrize("rows", [1, 3, 700])
@pytest.mark.parametrize("dt,rdt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_in_place(rows, dim, groups, dt, rdt):
    if rows * dim > 4_000_000 and rows > 3:
        rows = 4_200_000 // dim + 1  # still what takes few lanes for a part
    g = torch.Generator(device="cuda").manual_seed(dim)
    x, z = (torch.randn(rows, dim, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    res = (3 * torch.randn(rows, dim, generator=g, device="cuda")).to(DT[rdt])
    w = torch.rand(dim, generator=g, device="cuda").to(DT[dt])
    print("[gpu] norm in place", rows, dim, groups, dt, rdt, flush=True)
    for gate in (None, z):
        want, wu = ssu.add_rms_norm(x, w, res, gate, groups=groups)
        wx = ssu.add_rms_norm(x, w, None, gate, groups=groups)
        xs, rs = x.clone(), res.clone()
        y, u = ssu.add_rms_norm(xs, w, rs, gate, groups=groups, out=xs, residual_out=rs)
        assert y is xs and u is rs and torch.equal(y, want) and torch.equal(u, wu)
        xs = x.clone()
        assert torch.equal(ssu.add_rms_norm(xs, w, None, gate, groups=groups, out=xs), wx)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dim,groups", [(96, 1), (4128, 1), (40032, 1), (65568, 3)])
def test_residual_in_place_to_codes(dim, groups, fmt):
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn(5, dim, generator=g, device="cuda").bfloat16()
    res = 3 * torch.randn(5, dim, generator=g, device="cuda")
    w = torch.rand(dim, generator=g, device="cuda")
    (c, s), wu = ssu.add_rms_norm(x, w, res, groups=groups, out_format=fmt)
    rs = res.clone()
    (c2, s2), u = ssu.add_rms_norm(x, w, rs, groups=groups, out_format=fmt, residual_out=rs)
    assert u is rs and torch.equal(u, wu) and torch.equal(c, c2) and torch.equal(s, s2)
