"""Host-side checks of the layer operators' entry points: struct layouts, refusals
(every rule of include/ssu.h that the host checks, with the message naming it) and
empty calls, which launch nothing."""
import ctypes
import os
import subprocess

import pytest
import torch

import mamba_selective_state_amd as ssu
from mamba_selective_state_amd import layer as L
from mamba_selective_state_amd import ssu as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: every call here is refused or empty


def tdesc(shape, dtype, strides=None, ptr=FAKE):
    t = S.SsuTensor()
    t.data, t.dtype, t.ndim = ptr, dtype, len(shape)
    if strides is None:
        strides, acc = [], 1
        for s in reversed(shape):
            strides.insert(0, acc)
            acc *= s
    for i, (s, st) in enumerate(zip(shape, strides)):
        t.size[i], t.stride[i] = s, st
    return t


def test_struct_layout_matches_header(tmp_path):
    structs = {"ssu_norm_args_t": L.SsuNormArgs, "ssu_mx_linear_args_t": L.SsuMxLinearArgs,
               "ssu_logprob_args_t": L.SsuLogprobArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ssu.h"', "int main(void) {"]
    for cname, cls in structs.items():
        lines.append('printf("%s SIZEOF %%zu\\n", sizeof(%s));' % (cname, cname))
        for f, _ in cls._fields_:
            lines.append('printf("%s %s %%zu\\n", offsetof(%s, %s));' % (cname, f, cname, f))
    lines.append('printf("TOP MAX %d\\n", SSU_TOP_MAX);')
    lines.append("return 0; }")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "layout"), str(src)],
                   check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    assert got[("TOP", "MAX")] == L.TOP_MAX
    for cname, cls in structs.items():
        assert got[(cname, "SIZEOF")] == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert got[(cname, f)] == getattr(cls, f).offset, (cname, f)


def check(fn, *args):
    st = fn(*args)
    return st, S.ssu_last_error()


# ---------------------------------------------------------------- norm

def norm_args(rows=0, dim=64, groups=1, fmt=L.FORMAT_SAME, dt=S.BF16):
    a = L.SsuNormArgs()
    a.x = tdesc((rows, dim), dt)
    a.weight = tdesc((dim,), dt)
    if fmt == L.FORMAT_SAME:
        a.out = tdesc((rows, dim), dt)
    else:
        a.out = tdesc((rows, dim if fmt == L.FORMAT_MXFP8 else dim // 2), S.U8)
        a.out_scales = tdesc((rows, dim // 32), S.U8)
    a.groups, a.eps, a.out_format = groups, 1e-5, fmt
    return a


def norm(a):
    return check(S._lib.ssu_add_rms_norm, ctypes.byref(a), None)


def test_norm_empty_calls():
    for fmt in (L.FORMAT_SAME, L.FORMAT_MXFP4, L.FORMAT_MXFP8):
        assert norm(norm_args(fmt=fmt)) == (S.OK, "")
    assert norm(norm_args(rows=5, dim=0)) == (S.OK, "")


def _set(**kw):
    def f(a):
        for k, v in kw.items():
            setattr(a, k, v)
    return f


NORM_REFUSALS = [
    (_set(x=tdesc((4, 64, 1), S.BF16)), "x must be [rows, dim]"),
    (_set(x=tdesc((4, 64), S.I32)), "x must be f32, f16 or bf16"),
    (_set(x=tdesc((4, 64), S.BF16, (128, 2))), "x needs last stride 1"),
    (_set(x=tdesc((4, 64), S.BF16, (-64, 1))), "x has a negative stride"),
    (_set(x=tdesc((4, 64), S.BF16, ptr=FAKE + 1)), "x is not aligned"),
    (_set(weight=tdesc((63,), S.BF16)), "weight must be [64]"),
    (_set(weight=tdesc((64,), S.BF16, (2,))), "weight needs stride 1"),
    (_set(weight=tdesc((64,), S.F16)), "weight must have x's dtype or be f32"),
    (_set(weight=S.SsuTensor()), "weight is required"),
    (_set(gate=tdesc((4, 64), S.F32)), "gate must have x's dtype"),
    (_set(gate=tdesc((3, 64), S.BF16)), "gate must be [4, 64]"),
    (_set(residual=tdesc((4, 64), S.BF16)), "residual and residual_out go together"),
    (_set(residual=tdesc((4, 64), S.BF16), residual_out=tdesc((4, 64), S.F32)), "both have x's dtype or both be f32"),
    (_set(residual=tdesc((4, 64), S.F16), residual_out=tdesc((4, 64), S.F16)), "both have x's dtype or both be f32"),
    (_set(residual=tdesc((4, 64), S.F32), residual_out=tdesc((4, 64), S.F32, (32, 1))), "residual_out has overlapping rows"),
    (_set(out=S.SsuTensor()), "out is required"),
    (_set(out=tdesc((4, 64), S.F32)), "out must have x's dtype"),
    (_set(out=tdesc((4, 64), S.BF16, (0, 1))), "out has overlapping rows"),
    (_set(out_scales=tdesc((4, 2), S.U8)), "out_scales belongs to the MX formats"),
    (_set(groups=0), "groups must divide dim"),
    (_set(groups=3), "groups must divide dim"),
    (_set(eps=-1.0), "eps must be finite"),
    (_set(eps=float("nan")), "eps must be finite"),
]


@pytest.mark.parametrize("change,words", NORM_REFUSALS, ids=[w for _, w in NORM_REFUSALS])
def test_norm_refusals(change, words):
    a = norm_args(rows=4)
    change(a)
    st, msg = norm(a)
    assert st == S.ERR_VALUE and words in msg, msg


def test_norm_mx_refusals():
    a = norm_args(rows=4, dim=96, groups=2, fmt=L.FORMAT_MXFP8)
    assert norm(a)[0] == S.ERR_VALUE and "multiple of 32" in S.ssu_last_error()
    a = norm_args(rows=4, fmt=L.FORMAT_MXFP8)
    a.out_scales = S.SsuTensor()
    assert norm(a) == (S.ERR_VALUE, "out_scales is required")
    a = norm_args(rows=4, fmt=L.FORMAT_MXFP4)
    a.out = tdesc((4, 32), S.U8, (40, 1))
    assert norm(a) == (S.ERR_VALUE, "out must be contiguous")
    a = norm_args(rows=4, fmt=L.FORMAT_MXFP8)
    a.out.data = FAKE + 4
    assert norm(a) == (S.ERR_VALUE, "out must be 8-byte aligned")
    a = norm_args(rows=4)
    a.out_format = 7
    assert norm(a)[0] == S.ERR_NOT_IMPLEMENTED
    assert S._lib.ssu_add_rms_norm(None, None) == S.ERR_VALUE


# ---------------------------------------------------------------- MX quantisation and product

def quantize(src, codes, scales, fmt):
    return check(S._lib.ssu_mx_quantize, ctypes.byref(src), ctypes.byref(codes), ctypes.byref(scales), fmt, None)


def test_mx_quantize_empty_and_refusals():
    u8 = lambda *s: tdesc(s, S.U8)  # noqa: E731
    assert quantize(tdesc((0, 64), S.F16), u8(0, 32), u8(0, 2), L.FORMAT_MXFP4) == (S.OK, "")
    assert quantize(tdesc((3, 0), S.F16), u8(3, 0), u8(3, 0), L.FORMAT_MXFP8) == (S.OK, "")
    for src, codes, scales, fmt, words in (
            (tdesc((2, 48), S.F16), u8(2, 24), u8(2, 1), L.FORMAT_MXFP4, "multiple of 32"),
            (tdesc((2, 64), S.U8), u8(2, 32), u8(2, 2), L.FORMAT_MXFP4, "src must be [rows, k]"),
            (tdesc((64,), S.F16), u8(2, 32), u8(2, 2), L.FORMAT_MXFP4, "src must be [rows, k]"),
            (tdesc((2, 64), S.F16), u8(2, 64), u8(2, 2), L.FORMAT_MXFP4, "codes must be [2, 32]"),
            (tdesc((2, 64), S.F16), u8(2, 64), u8(2, 4), L.FORMAT_MXFP8, "scales must be [2, 2]"),
            (tdesc((2, 64), S.F16), tdesc((2, 64), S.U8, (80, 1)), u8(2, 2), L.FORMAT_MXFP8, "codes must be contiguous"),
            (tdesc((2, 64), S.F16), tdesc((2, 64), S.I32), u8(2, 2), L.FORMAT_MXFP8, "must be u8")):
        st, msg = quantize(src, codes, scales, fmt)
        assert st == S.ERR_VALUE and words in msg, msg
    assert quantize(tdesc((2, 64), S.F16), u8(2, 64), u8(2, 2), 5)[0] == S.ERR_NOT_IMPLEMENTED


def linear_args(m=0, n=48, k=64, fmt=L.FORMAT_MXFP8, x_dtype=S.BF16):
    a = L.SsuMxLinearArgs()
    if x_dtype == S.U8:
        a.x = tdesc((m, k if fmt == L.FORMAT_MXFP8 else k // 2), S.U8)
        a.x_scale = tdesc((m, k // 32), S.U8)
    else:
        a.x = tdesc((m, k), x_dtype)
    a.w = tdesc((n, k // 2), S.U8)
    a.w_scale = tdesc((n, k // 32), S.U8)
    a.out = tdesc((m, n), S.BF16)
    a.x_format = fmt
    return a


def linear(a, ws=None, nbytes=0):
    return check(S._lib.ssu_mx_linear, ctypes.byref(a), ws, nbytes, None)


def test_linear_empty_calls():
    assert linear(linear_args()) == (S.OK, "")
    assert linear(linear_args(x_dtype=S.U8)) == (S.OK, "")
    assert linear(linear_args(m=3, n=0)) == (S.OK, "")


LINEAR_REFUSALS = [
    (_set(w=tdesc((48, 32, 1), S.U8)), "must be 2-D"),
    (_set(w=tdesc((48, 40), S.U8)), "k must be a multiple of 32"),
    (_set(w=tdesc((48, 32), S.I32)), "w must be u8 codes"),
    (_set(w=tdesc((48, 32), S.U8, (40, 1))), "16-byte aligned base and row stride"),
    (_set(w=tdesc((48, 32), S.U8, ptr=FAKE + 8)), "16-byte aligned base and row stride"),
    (_set(w_scale=S.SsuTensor()), "w_scale must be given, as u8"),
    (_set(w_scale=tdesc((48, 3), S.U8)), "w_scale must be [48, 2]"),
    (_set(x=tdesc((4, 96), S.BF16)), "x must be [4, 64]"),
    (_set(x=tdesc((4, 64), S.U8)), "x_scale must be given"),
    (_set(x=tdesc((4, 64), S.I32)), "x must be u8 codes"),
    (_set(x_scale=tdesc((4, 2), S.U8)), "x_scale belongs to u8 codes"),
    (_set(out=tdesc((4, 47), S.BF16)), "out must be [4, 48]"),
    (_set(out=tdesc((4, 48), S.U8)), "out must be f32, f16 or bf16"),
    (_set(out=tdesc((4, 48), S.BF16, (24, 1))), "out has overlapping rows"),
    (_set(bias=tdesc((48,), S.F16)), "bias must be f32 or have out's dtype"),
    (_set(bias=tdesc((47,), S.F32)), "bias must be [48]"),
]


@pytest.mark.parametrize("change,words", LINEAR_REFUSALS, ids=[w for _, w in LINEAR_REFUSALS])
def test_linear_refusals(change, words):
    a = linear_args(m=4)
    change(a)
    st, msg = linear(a, FAKE, 1 << 20)
    assert st == S.ERR_VALUE and words in msg, msg


def test_linear_workspace_refusals():
    a = linear_args(m=4)
    need = S._lib.ssu_mx_linear_workspace_bytes(ctypes.byref(a))
    if need:
        for ws, nbytes in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
            st, msg = linear(a, ws, nbytes)
            assert st == S.ERR_VALUE and "workspace" in msg
    a.x_format = 0
    assert linear(a)[0] == S.ERR_NOT_IMPLEMENTED
    assert S._lib.ssu_mx_linear(None, None, 0, None) == S.ERR_VALUE
    assert S._lib.ssu_mx_linear_workspace_bytes(None) == 0


# ---------------------------------------------------------------- token log probabilities

def logprob_args(rows=0, vocab=100, top=3):
    a = L.SsuLogprobArgs()
    a.logits = tdesc((rows, vocab), S.BF16)
    a.tokens = tdesc((rows,), S.I64)
    a.logprob, a.entropy, a.rank = tdesc((rows,), S.F32), tdesc((rows,), S.F32), tdesc((rows,), S.I32)
    if top:
        a.top_tokens, a.top_logprobs = tdesc((rows, top), S.I32), tdesc((rows, top), S.F32)
    return a


def logprobs(a, ws=FAKE, nbytes=1 << 40):
    return check(S._lib.ssu_token_logprobs, ctypes.byref(a), ws, nbytes, None)


def test_logprob_empty_calls():
    assert logprobs(logprob_args()) == (S.OK, "")
    assert logprobs(logprob_args(top=0)) == (S.OK, "")


LOGPROB_REFUSALS = [
    (_set(logits=tdesc((4,), S.BF16)), "logits must be [rows, vocab]"),
    (_set(logits=tdesc((4, 100), S.I64)), "logits must be [rows, vocab]"),
    (_set(logits=tdesc((4, 100), S.BF16, (200, 2))), "logits needs last stride 1"),
    (_set(tokens=tdesc((4,), S.F32)), "tokens must be i32 or i64"),
    (_set(tokens=tdesc((3,), S.I64)), "tokens must be [4]"),
    (_set(mask=tdesc((4, 3), S.I32)), "mask must be [4, 4]"),
    (_set(mask=tdesc((4, 4), S.U8)), "mask must be i32"),
    (_set(temperature=tdesc((4,), S.BF16)), "temperature must be f32"),
    (_set(temperature=tdesc((4, 1), S.F32)), "temperature must be [4]"),
    (_set(logprob=tdesc((4,), S.BF16)), "logprob and entropy must be f32"),
    (_set(entropy=tdesc((4,), S.F32, (2,))), "entropy needs stride 1"),
    (_set(rank=tdesc((4,), S.I64)), "rank i32"),
    (_set(top_tokens=S.SsuTensor()), "go together"),
    (_set(top_tokens=tdesc((4, 3), S.I64)), "top_tokens must be i32"),
    (_set(top_logprobs=tdesc((4, 2), S.F32)), "top_logprobs must be [4, 3]"),
    (_set(top_tokens=tdesc((4, 3), S.I32, (6, 1))), "top_tokens must be contiguous"),
]


@pytest.mark.parametrize("change,words", LOGPROB_REFUSALS, ids=[w for _, w in LOGPROB_REFUSALS])
def test_logprob_refusals(change, words):
    a = logprob_args(rows=4)
    change(a)
    st, msg = logprobs(a)
    assert st == S.ERR_VALUE and words in msg, msg


def test_logprob_top_limit_and_null():
    st, msg = logprobs(logprob_args(rows=4, top=L.TOP_MAX + 1))
    assert st == S.ERR_NOT_IMPLEMENTED and "top must be at most" in msg
    assert S._lib.ssu_token_logprobs(None, None, 0, None) == S.ERR_VALUE


# ---------------------------------------------------------------- the Python functions

def test_python_functions_refuse():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ssu.add_rms_norm(x, torch.ones(64, dtype=torch.bfloat16), out=torch.empty_like(x))
    with pytest.raises(NotImplementedError, match="mxfp8"):
        ssu.add_rms_norm(x, torch.ones(64, dtype=torch.bfloat16), out_format="fp8")
    with pytest.raises(NotImplementedError, match="mxfp8"):
        ssu.mx_quantize(x, "int8")
    with pytest.raises(ValueError, match="collapse"):
        L._rows(torch.zeros(4, 6, 8).transpose(0, 1), "x")
    assert L._rows(torch.zeros(8), "x").shape == (1, 8)
    assert L._rows(torch.zeros(2, 3, 8), "x").shape == (6, 8)
