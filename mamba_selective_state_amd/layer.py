"""Python binding of the layer operators of libssu (include/ssu.h, "The layer
around the state update"): argument marshalling only, like ssu.py.

Low level, same names as the C ABI: ssu_add_rms_norm, ssu_mx_quantize,
ssu_mx_linear, ssu_token_logprobs. High level: add_rms_norm, mx_quantize,
mx_linear and token_logprobs, which take torch tensors and allocate what they
return; the marshalling of the three that a decode step calls is in C++
(csrc/ssu_torch.cpp), since their kernels take no longer than it takes in
Python. That module, which is bound to the torch it was built with, is loaded by
the first call of one of them; without it the call raises ImportError.
"""
import collections
import ctypes

import torch

from .ssu import OK, SsuError, SsuTensor, _lib, _raise, tensor_desc

FORMAT_SAME, FORMAT_MXFP4, FORMAT_MXFP8 = 0, 4, 8
TOP_MAX = 32  # SSU_TOP_MAX
_FORMATS = {"mxfp4": FORMAT_MXFP4, "mxfp8": FORMAT_MXFP8}


class SsuNormArgs(ctypes.Structure):
    _fields_ = [(n, SsuTensor) for n in
                ("x", "weight", "residual", "gate", "out", "out_scales", "residual_out")] + [
        ("groups", ctypes.c_int64), ("eps", ctypes.c_float), ("out_format", ctypes.c_int32)]


class SsuMxLinearArgs(ctypes.Structure):
    _fields_ = [(n, SsuTensor) for n in ("x", "x_scale", "w", "w_scale", "bias", "out")] + [
        ("x_format", ctypes.c_int32)]


class SsuLogprobArgs(ctypes.Structure):
    _fields_ = [(n, SsuTensor) for n in
                ("logits", "tokens", "mask", "temperature", "logprob", "entropy", "rank",
                 "top_tokens", "top_logprobs")]


_lib.ssu_add_rms_norm.argtypes = [ctypes.POINTER(SsuNormArgs), ctypes.c_void_p]
_lib.ssu_add_rms_norm.restype = ctypes.c_int
_lib.ssu_mx_quantize.argtypes = [ctypes.POINTER(SsuTensor)] * 3 + [ctypes.c_int32, ctypes.c_void_p]
_lib.ssu_mx_quantize.restype = ctypes.c_int
_lib.ssu_mx_linear_workspace_bytes.argtypes = [ctypes.POINTER(SsuMxLinearArgs)]
_lib.ssu_mx_linear_workspace_bytes.restype = ctypes.c_int64
_lib.ssu_mx_linear.argtypes = [ctypes.POINTER(SsuMxLinearArgs), ctypes.c_void_p, ctypes.c_int64,
                               ctypes.c_void_p]
_lib.ssu_mx_linear.restype = ctypes.c_int
_lib.ssu_token_logprobs_workspace_bytes.argtypes = [ctypes.POINTER(SsuLogprobArgs)]
_lib.ssu_token_logprobs_workspace_bytes.restype = ctypes.c_int64
_lib.ssu_token_logprobs.argtypes = [ctypes.POINTER(SsuLogprobArgs), ctypes.c_void_p, ctypes.c_int64,
                                    ctypes.c_void_p]
_lib.ssu_token_logprobs.restype = ctypes.c_int


_module = None


def _native():
    global _module
    if _module is None:
        try:
            from . import _ssu_torch
        except ImportError as e:
            raise ImportError("_ssu_torch.so is missing or was built for another torch: build the "
                              "package again (%s)" % e) from e
        _ssu_torch.set_error_type(SsuError)
        _module = _ssu_torch
    return _module


def _stream_of(t):
    """The handle of the current stream of a tensor's GPU (0 for a tensor that has none: the
    operators refuse it)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if t.is_cuda else 0


def _stream(stream):
    return torch.cuda.current_stream().cuda_stream if stream is None else stream


def ssu_add_rms_norm(args, stream=None):
    """Enqueue one RMS norm (include/ssu.h ssu_add_rms_norm)."""
    st = _lib.ssu_add_rms_norm(ctypes.byref(args), _stream(stream))
    if st != OK:
        _raise(st, "ssu_add_rms_norm")


def ssu_mx_quantize(src, codes, scales, out_format, stream=None):
    """Enqueue an MX quantisation of rows (include/ssu.h ssu_mx_quantize); the
    tensors are SsuTensor descriptors."""
    st = _lib.ssu_mx_quantize(ctypes.byref(src), ctypes.byref(codes), ctypes.byref(scales),
                              out_format, _stream(stream))
    if st != OK:
        _raise(st, "ssu_mx_quantize")


def ssu_mx_linear_workspace_bytes(args):
    return _lib.ssu_mx_linear_workspace_bytes(ctypes.byref(args))


def ssu_mx_linear(args, workspace=None, workspace_bytes=0, stream=None):
    """Enqueue a product with MXFP4 weights (include/ssu.h ssu_mx_linear)."""
    st = _lib.ssu_mx_linear(ctypes.byref(args), workspace, workspace_bytes, _stream(stream))
    if st != OK:
        _raise(st, "ssu_mx_linear")


def ssu_token_logprobs_workspace_bytes(args):
    return _lib.ssu_token_logprobs_workspace_bytes(ctypes.byref(args))


def ssu_token_logprobs(args, workspace=None, workspace_bytes=0, stream=None):
    """Enqueue token log probabilities (include/ssu.h ssu_token_logprobs)."""
    st = _lib.ssu_token_logprobs(ctypes.byref(args), workspace, workspace_bytes, _stream(stream))
    if st != OK:
        _raise(st, "ssu_token_logprobs")


def _format(name):
    f = _FORMATS.get(name)
    if f is None:
        raise NotImplementedError("format must be 'mxfp8' or 'mxfp4', got %r" % (name,))
    return f


def _rows(t, name):
    """[..., k] as [rows, k] without a copy."""
    if t is None or t.dim() == 2:
        return t
    if t.dim() == 0:
        raise ValueError("%s must have at least one dimension" % name)
    if t.dim() == 1:
        return t.unsqueeze(0)
    n = 1
    for s in t.shape[:-1]:
        n *= s
    try:
        return t.view(n, t.shape[-1])
    except RuntimeError:
        raise ValueError("%s: its leading dimensions must collapse to rows of one stride" % name)


def _mx_shapes(shape, fmt):
    lead, k = tuple(shape[:-1]), shape[-1]
    return lead + (k // 2 if fmt == FORMAT_MXFP4 else k,), lead + (k // 32,)


def make_norm_args(x, weight, out, out_scales=None, residual=None, residual_out=None, gate=None,
                   groups=1, eps=1e-5, out_format=FORMAT_SAME):
    """SsuNormArgs of 2-D tensors; the outputs must be given."""
    a = SsuNormArgs()
    for name, t in (("x", x), ("weight", weight), ("residual", residual), ("gate", gate),
                    ("out", out), ("out_scales", out_scales), ("residual_out", residual_out)):
        if t is not None:
            setattr(a, name, tensor_desc(t, x.device))
    a.groups, a.eps, a.out_format = groups, eps, out_format
    return a


def add_rms_norm(x, weight, residual=None, gate=None, groups=1, eps=1e-5, out_format=None, out=None,
                 out_scales=None, residual_out=None):
    """RMS norm over `groups` equal parts of each row of u = x * silu(gate) +
    residual (gate and residual optional), times `weight`.

    x, gate, residual [..., dim]; weight [dim] in x's dtype or float32; residual
    in x's dtype or float32. out_format None gives the result in x's dtype;
    "mxfp8" or "mxfp4" gives the pair (codes, scales) that mx_linear takes, uint8
    [..., dim] (or [..., dim / 2]) and [..., dim / 32]. With a residual the
    return value is (result, residual_out), residual_out = u in the residual's
    dtype. Outputs are allocated unless given; residual_out may be residual
    and out may be x. u is not rounded before the norm."""
    fmt = FORMAT_SAME if out_format is None else _format(out_format)
    y, scales, u = _native().add_rms_norm(x, weight, residual, gate, groups, eps, fmt, out,
                                          out_scales, residual_out, _stream_of(x))
    if scales is not None:
        y = (y, scales)
    return y if residual is None else (y, u)


def mx_quantize(x, out_format="mxfp4", codes=None, scales=None):
    """MXFP4 or MXFP8 of the rows of x [..., k] (float32, float16 or bfloat16,
    k a multiple of 32): a power-of-two scale byte per 32 values and E2M1 codes
    two a byte or E4M3 codes. A block that holds an infinity or a NaN gets the
    scale byte 0xFF and stands for NaNs. Returns (codes, scales)."""
    fmt = _format(out_format)
    cs, ss = _mx_shapes(x.shape, fmt) if x.dim() else ((0,), (0,))
    if codes is None:
        codes = torch.empty(cs, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(ss, dtype=torch.uint8, device=x.device)
    dev = x.device
    args = (tensor_desc(_rows(x, "x"), dev), tensor_desc(_rows(codes, "codes"), dev),
            tensor_desc(_rows(scales, "scales"), dev), fmt, _stream_of(x))
    with torch.cuda.device(dev):  # the default stream's handle is the current GPU's
        ssu_mx_quantize(*args)
    return codes, scales


def make_mx_linear_args(x, w, w_scale, out, x_scale=None, bias=None, x_format=FORMAT_MXFP8):
    """SsuMxLinearArgs of 2-D tensors; `out` must be given."""
    a = SsuMxLinearArgs()
    for name, t in (("x", x), ("x_scale", x_scale), ("w", w), ("w_scale", w_scale), ("bias", bias),
                    ("out", out)):
        if t is not None:
            setattr(a, name, tensor_desc(t, x.device))
    a.x_format = x_format
    return a


def mx_linear(x, weight, weight_scale, bias=None, activation="mxfp8", out=None, out_dtype=None):
    """x weight^T + bias with MXFP4 weights (uint8 codes [n, k / 2] and scales
    [n, k / 32], as mx_quantize makes them) and 8- or 4-bit activations.

    x is a float tensor [..., k], quantised in the call to `activation`
    ("mxfp8" or "mxfp4"), or a pair (codes, scales) from add_rms_norm or mx_quantize
    (its format is taken from its width). The result [..., n] has out_dtype
    (default: x's dtype, bfloat16 for a pair; `out`'s, if that is given); sums are kept in
    float32 and rounded once."""
    x_scale = None
    if isinstance(x, (tuple, list)):
        x, x_scale = x
        four = x.shape[-1] == weight.shape[-1]
        fmt = FORMAT_MXFP4 if four else FORMAT_MXFP8
    else:
        fmt = _format(activation)
    like = x if x_scale is None else None  # of the result's dtype; None: bfloat16
    if out is not None:
        if out_dtype is not None and out_dtype != out.dtype:
            raise ValueError("out_dtype is %s, out has %s" % (out_dtype, out.dtype))
    elif out_dtype is not None and out_dtype != (x.dtype if like is x else torch.bfloat16):
        out = torch.empty(x.shape[:-1] + weight.shape[:1], dtype=out_dtype, device=x.device)
    return _native().mx_linear(x, x_scale, weight, weight_scale, bias, fmt, out, like, _stream_of(x))


TokenLogprobs = collections.namedtuple(
    "TokenLogprobs", ("logprob", "entropy", "rank", "top_tokens", "top_logprobs"))


def make_logprob_args(logits, tokens, logprob, entropy, rank, top_tokens=None, top_logprobs=None,
                      mask=None, temperature=None):
    """SsuLogprobArgs; the outputs must be given."""
    a = SsuLogprobArgs()
    for name, t in (("logits", logits), ("tokens", tokens), ("mask", mask),
                    ("temperature", temperature), ("logprob", logprob), ("entropy", entropy),
                    ("rank", rank), ("top_tokens", top_tokens), ("top_logprobs", top_logprobs)):
        if t is not None:
            setattr(a, name, tensor_desc(t, logits.device))
    return a


def token_logprobs(logits, tokens, top=0, mask=None, temperature=None):
    """Log probabilities of one given token per row of logits [rows, vocab], with
    the row's entropy, the token's rank (how many allowed tokens stand before
    it: a larger logit, or an equal one at a lower index) and the `top` first
    alternatives with their log probabilities.

    mask: int32 [rows, ceil(vocab / 32)] (or one row of it, shared by all),
    bit i of word j allowing token 32 j + i; temperature: float32 [rows]. A
    token that is not allowed has log probability -inf and rank -1; missing
    alternatives are -1 and -inf. Returns a TokenLogprobs of float32 logprob and
    entropy, int32 rank, and int32 top_tokens and float32 top_logprobs
    [rows, top] (None without top)."""
    return TokenLogprobs(*_native().token_logprobs(logits, tokens, mask, temperature, top,
                                                   _stream_of(logits)))
