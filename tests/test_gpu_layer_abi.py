"""The layer operators through their C entry points (ssu_add_rms_norm, ssu_mx_linear,
ssu_token_logprobs, with make_*_args): the results of the Python functions bit for bit, with a workspace of
exactly the size asked for between guards."""
import pytest
import torch

import layer_ref as R
import mamba_selective_state_amd as ssu
from mamba_selective_state_amd import layer as L

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


class Guarded:
    """`need` bytes of device memory between two guards."""

    def __init__(self, need, zeroed=0):
        self.need = need
        self.all = torch.full((need + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        assert self.all.data_ptr() % 256 == 0
        self.all[GUARD:GUARD + min(zeroed, need)] = 0
        self.ptr = self.all.data_ptr() + GUARD if need else None

    def check(self):
        torch.cuda.synchronize()
        assert (self.all[:GUARD] == 0xA5).all() and (self.all[GUARD + self.need:] == 0xA5).all()


@pytest.mark.parametrize("fmt", [L.FORMAT_SAME, L.FORMAT_MXFP8, L.FORMAT_MXFP4])
@pytest.mark.parametrize("residual,gate", [(False, True), (True, False)])
def test_norm(fmt, residual, gate):
    g = torch.Generator().manual_seed(fmt)
    x, res, z = ((torch.randn(9, 768, generator=g) * s).bfloat16().cuda() for s in (1, 3, 2))
    w = torch.rand(768, generator=g).cuda()
    cols = {L.FORMAT_SAME: 768, L.FORMAT_MXFP8: 768, L.FORMAT_MXFP4: 384}[fmt]
    out = torch.empty(9, cols, dtype=torch.uint8 if fmt else torch.bfloat16, device="cuda")
    scales = torch.empty(9, 24, dtype=torch.uint8, device="cuda") if fmt else None
    u = torch.empty_like(res) if residual else None
    a = ssu.make_norm_args(x, w, out, scales, res if residual else None, u, z if gate else None, 3, 1e-4, fmt)
    print("[gpu] abi norm", fmt, flush=True)
    ssu.ssu_add_rms_norm(a)
    want = ssu.add_rms_norm(x, w, res if residual else None, z if gate else None, groups=3, eps=1e-4,
                            out_format={0: None, 8: "mxfp8", 4: "mxfp4"}[fmt])
    if residual:
        want, wu = want
        assert torch.equal(u, wu)
    assert torch.equal(out, want[0] if fmt else want) and (not fmt or torch.equal(scales, want[1]))


# streaming with codes made in a launch before, small tiles, middle ones, the large one and its last round
@pytest.mark.parametrize("m,n,k", [(3, 40, 96), (9, 100, 1056), (40, 520, 1056), (64, 2048, 512), (1100, 2080, 1312), (2100, 4100, 160), (4347, 4001, 96)])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("pair", [False, True])
def test_linear(m, n, k, fmt, pair):
    g = torch.Generator().manual_seed(m)
    x = torch.randn(m, k, generator=g).bfloat16().cuda()
    w, ws = ssu.mx_quantize(torch.randn(n, k, generator=g).cuda())
    codes = ssu.mx_quantize(x, fmt)
    want = ssu.mx_linear(codes if pair else x, w, ws, activation=fmt)
    out = torch.empty_like(want)
    a = ssu.make_mx_linear_args(codes[0] if pair else x, w, ws, out, codes[1] if pair else None, None,
                                L.FORMAT_MXFP8 if fmt == "mxfp8" else L.FORMAT_MXFP4)
    mem = Guarded(ssu.ssu_mx_linear_workspace_bytes(a))
    print("[gpu] abi linear", m, n, k, fmt, pair, mem.need, flush=True)
    for _ in range(2):
        out.fill_(7)
        ssu.ssu_mx_linear(a, mem.ptr, mem.need)
        mem.check()
        assert torch.equal(out, want)


@pytest.mark.parametrize("rows,vocab", [(1, 65536), (4, 50021), (255, 9000), (300, 5000)])
@pytest.mark.parametrize("top", [0, 5, 32])
def test_logprobs(rows, vocab, top):
    g = torch.Generator().manual_seed(rows)
    logits = (3 * torch.randn(rows, vocab, generator=g)).bfloat16().cuda()
    tokens = torch.randint(0, vocab, (rows,), generator=g).cuda()
    want = ssu.token_logprobs(logits, tokens, top)
    out = [torch.empty_like(t) if t is not None else None for t in want]
    a = ssu.make_logprob_args(logits, tokens, *out)
    mem = Guarded(ssu.ssu_token_logprobs_workspace_bytes(a), 2048)
    print("[gpu] abi logprobs", rows, vocab, top, mem.need, flush=True)
    for _ in range(3):
        for t in out[:3]:
            t.fill_(7)
        ssu.ssu_token_logprobs(a, mem.ptr, mem.need)
        mem.check()
        assert all(torch.equal(o, t) for o, t in zip(out, want) if t is not None)
        assert mem.need == 0 or (mem.all[GUARD:GUARD + 2048] == 0).all()  # as a call leaves them


def test_quantized_bytes():
    """MXFP4 code pairs bit for bit: the first value in the low half, a sign above three bits."""
    x = torch.randn(33, 256, generator=torch.Generator().manual_seed(5)) * 3
    codes, scales = ssu.mx_quantize(x.cuda(), "mxfp4")
    q, byte = R.quantize(x, "mxfp4")
    q = torch.where(q == 0, torch.zeros(()).double(), q)
    got = codes.cpu()
    zero = torch.tensor([8, 0], dtype=torch.uint8)  # -0 and 0 are one value
    low, high = got & 15, got >> 4
    low, high = (torch.where(h == zero[0], zero[1], h) for h in (low, high))
    assert torch.equal(low | (high << 4), R.encode_e2m1(q)) and torch.equal(scales.cpu(), byte)


def test_out_of_memory_is_torch_s():
    """An output that no GPU holds (the product's 360 GB): torch's own error, and the next call works."""
    x = torch.zeros(600_000, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(300_000, 16, dtype=torch.uint8, device="cuda")
    s = torch.zeros(300_000, 1, dtype=torch.uint8, device="cuda")
    print("[gpu] abi: more memory than there is", flush=True)
    with pytest.raises(torch.OutOfMemoryError):
        ssu.mx_linear(x, w, s)
    assert ssu.mx_linear(x[:40], w[:64], s[:64]).shape == (40, 64)
