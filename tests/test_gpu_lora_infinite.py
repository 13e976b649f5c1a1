"""add_lora with infinite weights, and with products beyond the range of float32: outputs are infinite, with the definition's sign, or
NaN where it is NaN; the others are off by what search_ref.lora allows."""
import math

import pytest
import torch

import mamba_selective_state_amd as ssu
import search_ref as S
from test_gpu_lora import DT, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def compare(c):
    print("[gpu] add_lora, infinite", tuple(c["x"].shape), c["x"].dtype, "a", tuple(c["a"].shape), flush=True)
    d = {k: v.cuda() for k, v in c.items()}
    got = ssu.add_lora(d["y"], d["x"], d["a"], d["b"], d["adapter"], d["scale"]).cpu()
    want, tol = S.lora(c["y"], c["x"], c["a"], c["b"], c["adapter"], c["scale"])
    as_type = want.to(got.dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isinf(got), torch.isinf(as_type))
    assert (got[torch.isinf(got)] == as_type[torch.isinf(got)]).all()
    fine = torch.isfinite(got)
    assert ((got.double() - want).abs() <= tol)[fine].all()
    return got


def signs_are_sure(c):
    """No h so near 0 that the float32 sums could give it the other sign."""
    for i in range(c["a"].shape[0]):
        x, w = c["x"][c["adapter"] == i].double(), c["a"][i].double()
        h, mag = x @ w.t(), x.abs() @ w.abs().t()
        if not bool((h.abs() > (x.shape[1] / 8 + 48) * 2.0 ** -23 * mag).all()):
            return False
    return True


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rank", [5, 16, 20, 64, 100])
@pytest.mark.parametrize("rows", [40, 300])
def test_infinite_weights(dt, rank, rows):
    c = next(c for c in (inputs(rows, 64, 150, rank, 3, dt, seed=s) for s in range(50)) if signs_are_sure(c))
    c["scale"][1] = -0.75
    for i in (1, 2):
        c["b"][i, 7, 2] = math.inf
        c["b"][i, 9, 0] = -math.inf
        c["b"][i, 130, 1], c["b"][i, 130, 4] = math.inf, math.inf  # NaN where the two h have other signs
        c["b"][i, 149] = -math.inf
    c["b"][2, 64, 3] = math.nan
    got = compare(c)
    assert torch.isinf(got[c["adapter"] == 1][:, [7, 9]]).all() and torch.isfinite(got[c["adapter"] == 0]).all()


def test_exact_h():
    """h of few bits: its second summand is 0."""
    for dt in DT:
        c = inputs(33, 32, 70, 16, 1, dt, none=0.0)
        c["x"] = torch.eye(33, 32).to(DT[dt])
        c["x"][32, 0] = 1
        c["a"] = (torch.randint(1, 4, c["a"].shape) * torch.where(torch.rand(c["a"].shape) < 0.5, -1, 1)).to(DT[dt])
        c["scale"][:] = 0.5
        c["b"][0, ::3, 5] = math.inf
        assert torch.isinf(compare(c)[:, ::3]).all()


def test_small_beside_large_h_in_f16():
    """An h far below f16's smallest part of the row's largest keeps its sign."""
    c = next(c for c in (inputs(40, 64, 50, 8, 1, "f16", seed=s, none=0.0) for s in range(50)) if signs_are_sure(c))
    c["a"] = (c["a"].float() * 1000).half()
    c["a"][0, 3] = 0
    c["a"][0, 3, 11] = 2.0 ** -24
    c["b"][0, ::7, 3] = math.inf
    assert torch.isinf(compare(c)[:, ::7]).all()


@pytest.mark.parametrize("rank", [16, 32])
@pytest.mark.parametrize("large,weight", [(1e6, 3e38), (1e30, 1e12)])
def test_products_beyond_float32(rank, large, weight):
    c = inputs(40, 64, 70, rank, 1, "bf16", none=0.0)
    c["x"] = c["x"] * large
    c["b"][0, 11] = 0
    c["b"][0, 11, 3] = weight
    c["b"][0, 65] = 0
    c["b"][0, 65, 1] = -weight
    h = c["x"].double() @ c["a"][0].double().t()
    assert (h[:, [1, 3]].abs() > 0.01 * large).all()
    assert torch.isinf(compare(c)[:, [11, 65]]).all()


def test_infinite_h_beside_large_ones_in_f16():
    """Beyond f16's own range, in a row that has an infinite one."""
    for rank in (8, 20):
        c = inputs(40, 64, 50, rank, 1, "f16", none=0.0)
        c["x"] = (c["x"].float() * 2000).half()
        c["a"] = (c["a"].float() * 300).half()
        c["b"] = (c["b"].float() * 2.0 ** -16).half()
        c["a"][0, 3, 5] = math.inf
        assert (c["x"][:, 5] != 0).all()
        assert torch.equal(torch.isinf(compare(c)), (c["b"][0, :, 3] != 0).expand(40, 50))
