"""Workspaces of the layer operators on the host: which calls need one, and that a missing, a short
or a misaligned one is refused before any launch."""
import ctypes

import pytest

from mamba_selective_state_amd import layer as L
from mamba_selective_state_amd import ssu as S
from test_layer_host import FAKE, check, linear_args, logprob_args

FMTS = [L.FORMAT_MXFP8, L.FORMAT_MXFP4]


def bad(need):
    return [(None, need), (None, 1 << 40), (FAKE, need - 1), (FAKE, 0), (FAKE + 16, need), (FAKE + 255, 1 << 40)]


def refused(fn, a, need):
    assert need > 0
    for ws, nbytes in bad(need):
        st, msg = check(fn, ctypes.byref(a), ws, nbytes, None)
        assert st == S.ERR_VALUE and "workspace must be 256-byte aligned and hold %d bytes" % need in msg, (ws, nbytes, msg)


# rows that are quantised for the streaming kernel, small and middle tiles, the large tile with a last round
@pytest.mark.parametrize("m,n,k", [(5, 48, 64), (16, 100, 4096), (17, 48, 64), (40, 520, 1056), (300, 4096, 512), (4347, 4001, 96)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("x_dtype", [S.BF16, S.F32, S.U8])
def test_linear(m, n, k, fmt, x_dtype):
    a = linear_args(m=m, n=n, k=k, fmt=fmt, x_dtype=x_dtype)
    need = S._lib.ssu_mx_linear_workspace_bytes(ctypes.byref(a))
    if m <= 16 and x_dtype == S.U8:  # scales are read where they are
        assert need == 0
        return
    codes = m * (k if fmt == L.FORMAT_MXFP8 else k // 2) if x_dtype != S.U8 else 0
    assert need >= codes + (m * (k // 32) if codes else 0)
    refused(S._lib.ssu_mx_linear, a, need)


@pytest.mark.parametrize("m", [1, 4])
@pytest.mark.parametrize("fmt", FMTS)
def test_linear_needs_none(m, fmt):
    assert S._lib.ssu_mx_linear_workspace_bytes(ctypes.byref(linear_args(m=m, fmt=fmt))) == 0


@pytest.mark.parametrize("rows,vocab", [(1, 65536), (4, 65536), (37, 50021), (255, 131072), (2, 4096)])
@pytest.mark.parametrize("top", [0, 1, 32])
def test_logprobs(rows, vocab, top):
    a = logprob_args(rows=rows, vocab=vocab, top=top)
    need = S._lib.ssu_token_logprobs_workspace_bytes(ctypes.byref(a))
    assert need > 2048
    refused(S._lib.ssu_token_logprobs, a, need)


@pytest.mark.parametrize("rows,vocab", [(0, 65536), (256, 131072), (2000, 65536), (3, 1000), (3, 0)])
def test_logprobs_need_none(rows, vocab):
    """Rows that one workgroup takes each."""
    assert S._lib.ssu_token_logprobs_workspace_bytes(ctypes.byref(logprob_args(rows=rows, vocab=vocab))) == 0
    assert S._lib.ssu_token_logprobs_workspace_bytes(None) == 0
