"""Sizes beyond what the operators of a beam search take.

reorder_states over more pools than one launch takes: a later launch that is too large is refused before the first one is
enqueued. The pointers are never dereferenced; without a GPU a launch would give another error."""
import pytest
import torch

import mamba_selective_state_amd as ssu
from mamba_selective_state_amd import ssu as S
from test_search_host import POOL, reorder, tables, tdesc

HUGE = tdesc((8, 2 ** 45), S.U8)           # 2^31 pieces of a slot
LARGE = tdesc((2 ** 18, 2 ** 22), S.U8)    # 256 pieces, of 2^17 requests


@pytest.mark.parametrize("first", [0, 63, 64, 65, 200])
def test_later_pools_too_large(first):
    for after in (0, 70):
        st, msg = reorder([POOL] * first + [HUGE] + [POOL] * after, *tables())
        assert st == S.ERR_NOT_IMPLEMENTED and "more rows or outputs than one launch takes" in msg, (st, msg)


@pytest.mark.parametrize("first", [0, 64, 130])
def test_too_many_requests_for_the_later_pools(first):
    tabs = [tdesc((2 ** 17, 2), S.I32, ptr=0x100000000 * (i + 1)) for i in range(3)]
    small = tdesc((2 ** 18, 4), S.U8)
    st, msg = reorder([small] * first + [LARGE], *tabs)
    assert st == S.ERR_NOT_IMPLEMENTED and "more rows or outputs than one launch takes" in msg, (st, msg)


@pytest.mark.parametrize("keep", [33, 2 ** 31, 2 ** 62])
def test_beam_select_refuses_keep_before_it_makes_outputs(keep):
    with pytest.raises(NotImplementedError, match="keep must be at most 32"):
        ssu.beam_select(torch.zeros(4, 8), torch.zeros(2, 2), keep)
