"""Python binding of beam search's operators of libssu (include/ssu.h, "Beam search
over a batch of requests").

Low level, same names as the C ABI: ssu_beam_select, ssu_reorder_states. High level:
beam_select and reorder_states, which take torch tensors; their marshalling is in C++
like that of the layer operators (layer.py).
"""
import collections
import ctypes

from .layer import _native, _stream, _stream_of
from .ssu import OK, SsuTensor, _lib, _raise, tensor_desc

BEAMS_MAX = 64  # SSU_BEAMS_MAX


class SsuBeamArgs(ctypes.Structure):
    _fields_ = [(n, SsuTensor) for n in
                ("logits", "scores", "finished", "mask", "out_scores", "out_parents", "out_tokens")] + [
        ("end_token", ctypes.c_int32)]


_lib.ssu_beam_select_workspace_bytes.argtypes = [ctypes.POINTER(SsuBeamArgs)]
_lib.ssu_beam_select_workspace_bytes.restype = ctypes.c_int64
_lib.ssu_beam_select.argtypes = [ctypes.POINTER(SsuBeamArgs), ctypes.c_void_p, ctypes.c_int64,
                                 ctypes.c_void_p]
_lib.ssu_beam_select.restype = ctypes.c_int
_lib.ssu_reorder_states.argtypes = [ctypes.POINTER(SsuTensor), ctypes.c_int32] + [
    ctypes.POINTER(SsuTensor)] * 3 + [ctypes.c_void_p]
_lib.ssu_reorder_states.restype = ctypes.c_int


def ssu_beam_select_workspace_bytes(args):
    return _lib.ssu_beam_select_workspace_bytes(ctypes.byref(args))


def ssu_beam_select(args, workspace=None, workspace_bytes=0, stream=None):
    """Enqueue a choice of continuations (include/ssu.h ssu_beam_select)."""
    st = _lib.ssu_beam_select(ctypes.byref(args), workspace, workspace_bytes, _stream(stream))
    if st != OK:
        _raise(st, "ssu_beam_select")


def ssu_reorder_states(pools, slots, parents, out_slots, stream=None):
    """Enqueue a reordering of states (include/ssu.h ssu_reorder_states); `pools` is a
    sequence of SsuTensor descriptors, the others are descriptors."""
    array = (SsuTensor * max(1, len(pools)))(*pools)
    st = _lib.ssu_reorder_states(array, len(pools), ctypes.byref(slots), ctypes.byref(parents),
                                 ctypes.byref(out_slots), _stream(stream))
    if st != OK:
        _raise(st, "ssu_reorder_states")


BeamSelection = collections.namedtuple("BeamSelection", ("scores", "parents", "tokens"))


def make_beam_args(logits, scores, out_scores, out_parents, out_tokens, finished=None, end_token=0,
                   mask=None):
    """SsuBeamArgs; the outputs must be given, finished as uint8."""
    a = SsuBeamArgs()
    for name, t in (("logits", logits), ("scores", scores), ("finished", finished), ("mask", mask),
                    ("out_scores", out_scores), ("out_parents", out_parents), ("out_tokens", out_tokens)):
        if t is not None:
            setattr(a, name, tensor_desc(t, logits.device))
    a.end_token = end_token
    return a


def beam_select(logits, scores, keep, finished=None, end_token=0, mask=None):
    """The first `keep` continuations of every request's beams.

    logits [batch, beams, vocab] or [batch * beams, vocab] (float32, float16 or bfloat16), scores float32
    [batch, beams]: the log probabilities of the sequences so far. Token v after beam i scores scores[b, i] +
    log_softmax(logits[b, i])[v], over the tokens that `mask` allows (as for token_logprobs) and whose
    logits are above -inf. A beam whose `finished` (bool or uint8 [batch, beams]) is set goes on with end_token alone, at an
    unchanged score; one at -inf does not go on (a search begins with all but one there). keep is at most 32:
    twice the beams, say, where continuations by the end token are taken out afterwards.

    Returns a BeamSelection of float32 scores and int32 parents (beams) and tokens, all [batch, keep], best
    first, equal scores by beam, then token; -inf, -1 and -1 where there are no more. A NaN or +inf among
    a request's scores or the logits that count makes its scores NaN and the rest -1."""
    return BeamSelection(*_native().beam_select(logits, scores, keep, finished, end_token, mask,
                                                _stream_of(logits)))


def reorder_states(pools, slots, parents, out_slots=None):
    """Lets the sequences' states follow a choice of continuations.

    pools: a tensor [slots, ...], or a list of them (every layer's states and convolution states), of any dtype, each
    slot's elements contiguous. slots int32 or int64 [batch, beams]: the slots of the beams, as selective_state_update's
    state_batch_indices name them. parents [batch, beams]: the beam that each new one goes on from (of
    BeamSelection.parents, as many as there are beams). The first new beam of a parent keeps its slot; for every further one the
    parent's slot is copied to that of a beam that nothing goes on from. A new beam whose parent is none of [0, beams), such as
    -1, gets such a slot too, with what it holds. Returns the new beams' slots, in `out_slots` if that is given (not the
    memory of slots or parents)."""
    return _native().reorder_states(pools, slots, parents, out_slots, _stream_of(slots))
