"""Sizes at and past what the layer operators' kernels count in 32 bits: refused by name on the
host, before any launch. (A kernel rounds its indexes up to whole accesses, tiles and rounds of
them: sizes near 2^31 would turn them negative.)"""
import ctypes

import pytest

from mamba_selective_state_amd import layer as L
from mamba_selective_state_amd import ssu as S
from test_layer_host import FAKE, check, linear_args, logprob_args, norm_args, tdesc

INT_MAX = 2 ** 31 - 1
NEAR = [INT_MAX, INT_MAX - 1, INT_MAX - 8191, INT_MAX - 65535, INT_MAX + 1, 2 ** 33]


def down(v, unit):
    return v // unit * unit


@pytest.mark.parametrize("dim", NEAR)
@pytest.mark.parametrize("fmt", [L.FORMAT_SAME, L.FORMAT_MXFP8, L.FORMAT_MXFP4])
def test_norm(dim, fmt):
    a = norm_args(rows=1, dim=max(down(dim, 32), INT_MAX - 65535 + 31 & ~31), fmt=fmt)
    st, msg = check(S._lib.ssu_add_rms_norm, ctypes.byref(a), None)
    assert st == S.ERR_VALUE and "size out of range" in msg, msg


@pytest.mark.parametrize("k", NEAR)
@pytest.mark.parametrize("fmt", [L.FORMAT_MXFP8, L.FORMAT_MXFP4])
def test_quantize(k, fmt):
    k = max(down(k, 32), INT_MAX - 65535 + 31 & ~31)
    codes = tdesc((1, k if fmt == L.FORMAT_MXFP8 else k // 2), S.U8)
    st, msg = check(S._lib.ssu_mx_quantize, ctypes.byref(tdesc((1, k), S.F16)), ctypes.byref(codes),
                    ctypes.byref(tdesc((1, k // 32), S.U8)), fmt, None)
    assert st == S.ERR_NOT_IMPLEMENTED and "k too large" in msg, msg


@pytest.mark.parametrize("size", NEAR)
@pytest.mark.parametrize("which", ["m", "n", "k"])
@pytest.mark.parametrize("x_dtype", [S.BF16, S.U8])
def test_linear(which, size, x_dtype):
    size = max(down(size, 32), INT_MAX - 65535 + 31 & ~31)
    a = linear_args(**{"m": 40, "n": 48, "k": 64, "x_dtype": x_dtype, which: size})
    st, msg = check(S._lib.ssu_mx_linear, ctypes.byref(a), FAKE, 1 << 60, None)
    assert st == S.ERR_VALUE and "size out of range" in msg, msg


@pytest.mark.parametrize("size", NEAR)
def test_logprobs(size):
    a = logprob_args(rows=1, vocab=max(size, INT_MAX - 65535))
    st, msg = check(S._lib.ssu_token_logprobs, ctypes.byref(a), FAKE, 1 << 60, None)
    assert st == S.ERR_VALUE and "size out of range" in msg, msg


@pytest.mark.parametrize("rows,dim,groups", [(2 ** 26, 4, 1), (2 ** 27, 7, 1), (2 ** 25, 4, 2), (2 ** 28 + 16, 8, 1), (2 ** 24, 32768, 1)])
def test_norm_rows_of_one_launch(rows, dim, groups):
    """2^32 work items: a wave for each short part, 16 lanes up to 128 elements, a workgroup of 256
    from 4096 on."""
    a = norm_args(rows=rows, dim=dim, groups=groups)
    st, msg = check(S._lib.ssu_add_rms_norm, ctypes.byref(a), None)
    assert st == S.ERR_NOT_IMPLEMENTED and "one launch" in msg, msg


def test_logprob_rows_of_one_launch():
    a = logprob_args(rows=2 ** 24, vocab=100)
    st, msg = check(S._lib.ssu_token_logprobs, ctypes.byref(a), None, 0, None)
    assert st == S.ERR_NOT_IMPLEMENTED and "one launch" in msg, msg


def test_linear_outputs_of_one_launch():
    a = linear_args(m=2, n=2 ** 28, k=32)
    st, msg = check(S._lib.ssu_mx_linear, ctypes.byref(a), FAKE, 1 << 60, None)
    assert st == S.ERR_NOT_IMPLEMENTED and "one launch" in msg, msg
