"""Host-side checks of beam_select, reorder_states and add_lora: struct layouts, refusals (every rule of
include/ssu.h that the host checks, with the message naming it), empty calls, which launch nothing, and
workspaces. The pointers are never dereferenced: every call here is refused or empty."""
import ctypes
import os
import subprocess

import pytest
import torch

import mamba_selective_state_amd as ssu
from mamba_selective_state_amd import layer as L
from mamba_selective_state_amd import search as B
from mamba_selective_state_amd import ssu as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


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
    structs = {"ssu_lora_args_t": L.SsuLoraArgs, "ssu_beam_args_t": B.SsuBeamArgs}
    limits = {"SSU_BEAMS_MAX": B.BEAMS_MAX, "SSU_LORA_RANK_MAX": L.LORA_RANK_MAX, "SSU_LORA_ADAPTERS_MAX": L.LORA_ADAPTERS_MAX}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ssu.h"', "int main(void) {"]
    for cname, cls in structs.items():
        lines.append('printf("%s SIZEOF %%zu\\n", sizeof(%s));' % (cname, cname))
        for f, _ in cls._fields_:
            lines.append('printf("%s %s %%zu\\n", offsetof(%s, %s));' % (cname, f, cname, f))
    for name in limits:
        lines.append('printf("LIMIT %s %%d\\n", %s);' % (name, name))
    lines.append("return 0; }")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    got = {tuple(line.split()[:2]): int(line.split()[2]) for line in out.splitlines()}
    for name, v in limits.items():
        assert got[("LIMIT", name)] == v
    for cname, cls in structs.items():
        assert got[(cname, "SIZEOF")] == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert got[(cname, f)] == getattr(cls, f).offset, (cname, f)


def _set(**kw):
    def f(a):
        for k, v in kw.items():
            setattr(a, k, v)
    return f


def refused(fn, a, words, more=(None, 0, None)):
    st = fn(ctypes.byref(a), *more)
    msg = S.ssu_last_error()
    assert st in (S.ERR_VALUE, S.ERR_NOT_IMPLEMENTED) and words in msg, (st, msg)
    return st


# ---------------------------------------------------------------- add_lora

def lora_args(rows=4, k=64, n=48, rank=8, adapters=3, dt=S.BF16, fmt=L.FORMAT_SAME):
    a = L.SsuLoraArgs()
    if fmt == L.FORMAT_SAME:
        a.x = tdesc((rows, k), dt)
    else:
        a.x = tdesc((rows, k if fmt == L.FORMAT_MXFP8 else k // 2), S.U8)
        a.x_scale = tdesc((rows, k // 32), S.U8)
    a.a, a.b = tdesc((adapters, rank, k), dt), tdesc((adapters, n, rank), dt)
    a.adapter, a.scale, a.y = tdesc((rows,), S.I32), tdesc((adapters,), S.F32), tdesc((rows, n), dt)
    a.x_format = fmt
    return a


LORA_REFUSALS = [
    (_set(y=S.SsuTensor()), "y must be 2-D, a and b 3-D"),
    (_set(a=tdesc((24, 64), S.BF16)), "y must be 2-D, a and b 3-D"),
    (_set(b=tdesc((3, 48, 8), S.F16)), "a, b and y must have one dtype"),
    (_set(y=tdesc((4, 48), S.F32)), "a, b and y must have one dtype"),
    (_set(a=tdesc((3, 8, 64), S.U8)), "a, b and y must have one dtype"),
    (_set(x=tdesc((4, 64), S.F32)), "x must have a's dtype"),
    (_set(x=S.SsuTensor()), "x must have a's dtype"),  # absent: of no dtype
    (_set(x=tdesc((3, 64), S.BF16)), "x must be [4, 64]"),
    (_set(x=tdesc((4, 64), S.BF16, (1, 4))), "x needs last stride 1"),
    (_set(x=tdesc((4, 64), S.BF16, (-64, 1))), "x has a negative stride"),
    (_set(x=tdesc((4, 64), S.BF16, ptr=FAKE + 1)), "x is not aligned"),
    (_set(x_scale=tdesc((4, 2), S.U8)), "x_scale belongs to the MX formats"),
    (_set(a=tdesc((3, 8, 64), S.BF16, (512, 1, 8))), "a needs last stride 1"),
    (_set(a=tdesc((3, 8, 64), S.BF16, (-512, 64, 1))), "a has a negative stride"),
    (_set(a=tdesc((3, 129, 64), S.BF16)), "rank must be at most 128"),
    (_set(a=tdesc((4097, 8, 64), S.BF16)), "at most 4096 adapters"),
    (_set(b=tdesc((2, 48, 8), S.BF16)), "b must be [3, 48, 8]"),
    (_set(b=tdesc((3, 48, 7), S.BF16)), "b must be [3, 48, 8]"),
    (_set(b=tdesc((3, 48, 8), S.BF16, (384, 1, 48))), "b needs last stride 1"),
    (_set(b=tdesc((3, 48, 8), S.BF16, ptr=FAKE + 1)), "b is not aligned"),
    (_set(adapter=tdesc((4,), S.F32)), "adapter must be i32 or i64"),
    (_set(adapter=tdesc((5,), S.I32)), "adapter must be [4]"),
    (_set(adapter=tdesc((4,), S.I32, (-1,))), "adapter has a negative stride"),
    (_set(scale=tdesc((3,), S.BF16)), "scale must be f32"),
    (_set(scale=tdesc((4,), S.F32)), "scale must be [3]"),
    (_set(y=tdesc((4, 48), S.BF16, (24, 1))), "y has overlapping rows"),
    (_set(y=tdesc((4, 48), S.BF16, (0, 1))), "y has overlapping rows"),
    (_set(x_format=5), "x_format must be SAME, MXFP8 or MXFP4"),
    (lambda a: None, "workspace must be 256-byte aligned and hold"),
]


@pytest.mark.parametrize("change,words", LORA_REFUSALS, ids=[w for _, w in LORA_REFUSALS])
def test_lora_refusals(change, words):
    a = lora_args()
    change(a)
    refused(S._lib.ssu_add_lora, a, words)


def test_lora_refusals_of_codes():
    f8 = L.FORMAT_MXFP8
    fn = S._lib.ssu_add_lora
    refused(fn, lora_args(dt=S.F16, fmt=f8), "x of codes needs a, b and y in bf16")
    a = lora_args(k=40, fmt=f8)
    refused(fn, a, "k to be a multiple of 32")
    a = lora_args(fmt=f8)
    a.x_scale = S.SsuTensor()
    refused(fn, a, "x of codes and x_scale must be u8")
    a = lora_args(fmt=f8)
    a.x_scale = tdesc((4, 3), S.U8)
    refused(fn, a, "x_scale must be [4, 2]")
    a = lora_args(fmt=L.FORMAT_MXFP4)
    a.x = tdesc((4, 64), S.U8)
    refused(fn, a, "x must be [4, 32]")


def test_lora_empty_calls_and_workspace():
    fn, need = S._lib.ssu_add_lora, S._lib.ssu_add_lora_workspace_bytes
    for kw in ({"rows": 0}, {"n": 0}, {"k": 0}, {"rank": 0}, {"adapters": 0}):
        a = lora_args(**kw)
        assert (fn(ctypes.byref(a), None, 0, None), S.ssu_last_error()) == (S.OK, "")
    a = lora_args()
    bytes_ = need(ctypes.byref(a))
    assert bytes_ > 0
    refused(fn, a, "workspace", (ctypes.c_void_p(FAKE), bytes_ - 1, None))
    refused(fn, a, "workspace", (ctypes.c_void_p(FAKE + 16), bytes_, None))
    refused(fn, a, "workspace", (None, bytes_, None))
    assert S._lib.ssu_add_lora(None, None, 0, None) == S.ERR_VALUE
    # room for the rows' numbers and h, whatever the sizes
    for rows in (1, 2048, 2049, 100000):
        for rank, padded in ((1, 16), (17, 32), (64, 64), (65, 128)):
            assert need(ctypes.byref(lora_args(rows=rows, rank=rank))) >= rows * (4 + 4 * padded)


def test_lora_too_large_for_one_launch():
    """2^30 rows of 2^31 outputs: more tiles than one launch has numbers for."""
    a = lora_args(rows=2 ** 30, n=2 ** 31 - 70000)
    need = S._lib.ssu_add_lora_workspace_bytes(ctypes.byref(a))
    assert refused(S._lib.ssu_add_lora, a, "more rows or outputs than one launch takes", (ctypes.c_void_p(FAKE), need, None)) == S.ERR_NOT_IMPLEMENTED


# ---------------------------------------------------------------- beam_select

def beam_args(batch=2, beams=3, vocab=50, keep=4, dt=S.BF16):
    a = B.SsuBeamArgs()
    a.logits, a.scores = tdesc((batch * beams, vocab), dt), tdesc((batch, beams), S.F32)
    a.out_scores = tdesc((batch, keep), S.F32)
    a.out_parents, a.out_tokens = tdesc((batch, keep), S.I32), tdesc((batch, keep), S.I32)
    return a


BEAM_REFUSALS = [
    (_set(logits=S.SsuTensor()), "logits must be [batch * beams, vocab]"),
    (_set(logits=tdesc((6, 50), S.I32)), "logits must be [batch * beams, vocab]"),
    (_set(logits=tdesc((5, 50), S.BF16)), "logits must be [6, 50]"),
    (_set(logits=tdesc((6, 50), S.BF16, (1, 6))), "logits needs last stride 1"),
    (_set(logits=tdesc((6, 50), S.BF16, ptr=FAKE + 1)), "logits is not aligned"),
    (_set(scores=tdesc((6,), S.F32)), "scores must be [batch, beams], f32"),
    (_set(scores=tdesc((2, 3), S.F16)), "scores must be [batch, beams], f32"),
    (_set(scores=tdesc((2, 3), S.F32, (3, -1))), "scores has a negative stride"),
    (_set(scores=tdesc((2, 65), S.F32)), "beams must be 1 to 64"),
    (_set(scores=tdesc((2, 0), S.F32)), "beams must be 1 to 64"),
    (_set(finished=tdesc((2, 3), S.I32)), "finished must be u8"),
    (_set(finished=tdesc((2, 4), S.U8)), "finished must be [2, 3]"),
    (_set(finished=tdesc((2, 3), S.U8), end_token=50), "end_token must lie in the vocabulary"),
    (_set(finished=tdesc((2, 3), S.U8), end_token=-1), "end_token must lie in the vocabulary"),
    (_set(mask=tdesc((6, 2), S.U8)), "mask must be i32"),
    (_set(mask=tdesc((6, 1), S.I32)), "mask must be [6, 2]"),
    (_set(out_tokens=S.SsuTensor()), "out_tokens must be [batch, keep]"),
    (_set(out_tokens=tdesc((2, 33), S.I32)), "keep must be at most 32"),
    (_set(out_tokens=tdesc((2, 4), S.I64)), "out_scores must be f32, out_parents and out_tokens i32"),
    (_set(out_scores=tdesc((2, 5), S.F32)), "out_scores must be [2, 4]"),
    (_set(out_parents=tdesc((2, 4), S.I32, (8, 1))), "out_parents must be contiguous"),
    (lambda a: None, "workspace must be 256-byte aligned and hold"),
]


@pytest.mark.parametrize("change,words", BEAM_REFUSALS, ids=[w for _, w in BEAM_REFUSALS])
def test_beam_refusals(change, words):
    a = beam_args()
    change(a)
    refused(S._lib.ssu_beam_select, a, words)


def test_beam_empty_calls_and_workspace():
    fn, need = S._lib.ssu_beam_select, S._lib.ssu_beam_select_workspace_bytes
    for kw in ({"batch": 0}, {"keep": 0}):
        a = beam_args(**kw)
        assert (fn(ctypes.byref(a), None, 0, None), S.ssu_last_error()) == (S.OK, "")
    a = beam_args()
    bytes_ = need(ctypes.byref(a))
    refused(fn, a, "workspace", (ctypes.c_void_p(FAKE), bytes_ - 1, None))
    refused(fn, a, "workspace", (ctypes.c_void_p(FAKE + 8), bytes_, None))
    assert S._lib.ssu_beam_select(None, None, 0, None) == S.ERR_VALUE
    # a list of every row at least, and no more lists of a request than the second kernel has room for
    for batch, beams, vocab in ((1, 1, 5), (1, 64, 2 ** 20), (1, 3, 2 ** 24), (300, 7, 10 ** 5), (4, 64, 10 ** 6)):
        for keep in (1, 32):
            n = need(ctypes.byref(beam_args(batch, beams, vocab, keep)))
            assert batch * beams * (8 * keep + 8) <= n <= batch * max(512, beams) * (8 * keep + 8) + 256


# ---------------------------------------------------------------- reorder_states

def reorder(pools, slots, parents, out):
    array = (S.SsuTensor * max(1, len(pools)))(*pools)
    st = S._lib.ssu_reorder_states(array, len(pools), *(None if t is None else ctypes.byref(t) for t in (slots, parents, out)), None)
    return st, S.ssu_last_error()


def tables(**kw):
    t = {"slots": tdesc((2, 3), S.I32), "parents": tdesc((2, 3), S.I32, ptr=FAKE + 64), "out": tdesc((2, 3), S.I32, ptr=FAKE + 128)}
    t.update(kw)
    return t["slots"], t["parents"], t["out"]


POOL = tdesc((9, 4, 5), S.F32)
REORDER_REFUSALS = [
    ([POOL], tables(slots=None), "a tensor is NULL"),
    ([POOL], tables(slots=tdesc((6,), S.I32)), "slots must be [batch, beams]"),
    ([POOL], tables(slots=tdesc((2, 65), S.I32)), "beams must be 1 to 64"),
    ([POOL], tables(slots=tdesc((2, 3), S.F32)), "must be i32 or i64"),
    ([POOL], tables(parents=tdesc((2, 4), S.I32)), "parents must be [2, 3]"),
    ([POOL], tables(parents=tdesc((2, 3), S.I64, (-3, 1))), "parents has a negative stride"),
    ([POOL], tables(out=tdesc((3, 3), S.I32)), "out_slots must be [2, 3]"),
    ([POOL], tables(out=tdesc((2, 3), S.I32, (2, 1), ptr=FAKE + 128)), "out_slots has overlapping rows"),
    ([POOL], tables(out=tdesc((2, 3), S.I32)), "out_slots overlaps slots or parents"),
    ([POOL], tables(out=tdesc((2, 3), S.I32, ptr=FAKE + 64 - 20)), "out_slots overlaps slots or parents"),
    ([S.SsuTensor()], tables(), "pool 0 must be [slots, ...]"),
    ([POOL, tdesc((9, 4, 5), S.F32, (20, 1, 4))], tables(), "pool 1: a slot's elements must be contiguous"),
    ([POOL, POOL, tdesc((9, 4, 5), S.F32, (19, 5, 1))], tables(), "pool 2 has overlapping slots"),
    ([tdesc((9, 4), 9)], tables(), "pool 0 must be [slots, ...]"),
]


@pytest.mark.parametrize("pools,tabs,words", REORDER_REFUSALS, ids=range(len(REORDER_REFUSALS)))
def test_reorder_refusals(pools, tabs, words):
    st, msg = reorder(pools, *tabs)
    assert st in (S.ERR_VALUE, S.ERR_NOT_IMPLEMENTED) and words in msg, (st, msg)


def test_reorder_empty():
    empty = [tdesc((0, 3), S.I32, ptr=FAKE + 64 * i) for i in range(3)]
    assert reorder([POOL], *empty) == (S.OK, "")
    assert S._lib.ssu_reorder_states(None, 2, *(ctypes.byref(t) for t in tables()), None) == S.ERR_VALUE
    assert S._lib.ssu_reorder_states(None, -1, *(ctypes.byref(t) for t in tables()), None) == S.ERR_VALUE


# ---------------------------------------------------------------- the Python functions

def test_python_refusals_without_a_gpu():
    """Tensors on the CPU, and arguments of other kinds."""
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ssu.beam_select(x, torch.zeros(2, 2), 2)
    with pytest.raises(ValueError, match="GPU"):
        ssu.reorder_states([x], torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        ssu.add_lora(x, x, torch.zeros(1, 2, 8), torch.zeros(1, 8, 2), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="keep must not be negative"):
        ssu.beam_select(x, torch.zeros(2, 2), -1)
    with pytest.raises(ValueError, match="end_token"):
        ssu.beam_select(x, torch.zeros(2, 2), 2, end_token=2 ** 40)
    with pytest.raises(TypeError):
        ssu.beam_select(x, None, 2)
    with pytest.raises(TypeError):
        ssu.reorder_states("pool", torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        ssu.add_lora(x, x, None, None, None)
