"""Plain float64 forms of the layer operators (add_rms_norm, mx_quantize, mx_linear,
token_logprobs), on the CPU, written from their definitions in include/ssu.h."""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
EMAX = {"mxfp8": 8, "mxfp4": 2}
LARGEST = {"mxfp8": 448.0, "mxfp4": 6.0}
SMALLEST_EXP = {"mxfp8": -6, "mxfp4": 0}  # of a normal element
MANTISSA = {"mxfp8": 3, "mxfp4": 1}
# half an ulp of the largest relative size (unit roundoff)
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def norm(x, weight, residual=None, gate=None, groups=1, eps=1e-5):
    """(y, u, scale of the error): y and u in float64, and for every element the
    magnitude that its fp32 roundings are relative to."""
    v = x.double()
    if gate is not None:
        v = v * torch.sigmoid(gate.double()) * gate.double()
    mag = v.abs()
    u = v
    if residual is not None:
        u = v + residual.double()
        mag = mag + residual.double().abs()
    parts = u.reshape(u.shape[0], groups, -1)
    inv = 1.0 / torch.sqrt((parts ** 2).mean(-1, keepdim=True) + eps)
    y = (parts * inv).reshape(u.shape) * weight.double()
    size = (mag.reshape(parts.shape) * inv).reshape(u.shape) * weight.double().abs()
    return y, u, size


def step(v, fmt):
    """The distance between neighbouring values of the element format around v."""
    _, e = torch.frexp(v.abs())
    e = torch.clamp(e - 1, min=SMALLEST_EXP[fmt])
    return torch.ldexp(torch.ones_like(v), e - MANTISSA[fmt])


def quantize(x, fmt):
    """(values, scale bytes) of the rows of x in float64: the value that each code
    stands for over its scale, NaN in a block that is not finite."""
    b = x.double().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    _, e = torch.frexp(torch.where(bad | (amax == 0), torch.ones_like(amax), amax))
    k = torch.clamp(torch.where(amax == 0, torch.full_like(e, -126), e - 1 - EMAX[fmt]), -126, 127)
    # fp32 subnormals have no exponent of their own: the smallest scale
    k = torch.where(amax < 2.0 ** -126, torch.full_like(k, -126), k)
    v = torch.ldexp(b, -k)
    s = step(v, fmt)
    q = torch.clamp(torch.round(v / s) * s, -LARGEST[fmt], LARGEST[fmt])
    q = torch.where(bad, torch.full_like(q, math.nan), q)
    byte = torch.where(bad, torch.full_like(k, 255), k + 127)
    return q.reshape(x.shape), byte[..., 0].to(torch.uint8)


def decode(codes, scales, fmt):
    """The float64 values that codes and scales stand for."""
    codes, scales = codes.cpu(), scales.cpu()
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).double()
    else:
        table = torch.tensor(E2M1 + [-t for t in E2M1], dtype=torch.float64)
        v = table[torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).long()]
    x = torch.ldexp(torch.ones(scales.shape, dtype=torch.float64), scales.int() - 127)
    x = torch.where(scales == 255, torch.full_like(x, math.nan), x)
    return v * x.repeat_interleave(32, -1)


def encode_e2m1(values):
    """Code pairs of exact E2M1 values."""
    table = torch.tensor(E2M1, dtype=torch.float64)
    c = torch.searchsorted(table, values.abs().double().contiguous()).to(torch.uint8)
    c = c + torch.where(values < 0, 8, 0).to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def logprobs(logits, tokens, top=0, mask=None, temperature=None):
    """The five results for every row, in float64 and whole numbers."""
    rows, vocab = logits.shape
    out = {"logprob": [], "entropy": [], "rank": [], "top_tokens": [], "top_logprobs": []}
    for r in range(rows):
        raw = logits[r].double()
        listed = torch.ones(vocab, dtype=torch.bool)
        if mask is not None:
            at = torch.arange(vocab)
            listed = ((mask[r].long()[at // 32] >> (at % 32)) & 1) == 1
        temp = 1.0 if temperature is None else float(temperature[r])
        bad = not temp > 0 or bool((listed & ~(raw < math.inf)).any())
        ok = listed & (raw > -math.inf)
        t = int(tokens[r])
        if bad:
            out["logprob"].append(math.nan)
            out["entropy"].append(math.nan)
            out["rank"].append(-1)
            out["top_tokens"].append([-1] * top)
            out["top_logprobs"].append([math.nan] * top)
            continue
        ids = torch.nonzero(ok)[:, 0]
        l = raw[ids]
        l = (l - l.max()) / temp if len(ids) else l  # before the logarithm, which 1e38 would swallow
        logp = l - torch.log(torch.exp(l).sum())
        order = torch.sort(raw[ids], descending=True, stable=True).indices
        place = {int(ids[i]): n for n, i in enumerate(order.tolist())}
        where = {int(i): n for n, i in enumerate(ids.tolist())}
        out["entropy"].append(float(-(torch.exp(logp) * logp).sum()))
        out["logprob"].append(float(logp[where[t]]) if t in where else -math.inf)
        out["rank"].append(place.get(t, -1))
        first = order[:top].tolist()
        out["top_tokens"].append([int(ids[i]) for i in first] + [-1] * (top - len(first)))
        out["top_logprobs"].append([float(logp[i]) for i in first] + [-math.inf] * (top - len(first)))
    return {k: torch.tensor(v, dtype=torch.int32 if k in ("rank", "top_tokens") else torch.float64)
            for k, v in out.items()}
