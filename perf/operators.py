"""The cases by which the layer operators around the state update are measured: add_rms_norm, mx_linear and
token_logprobs (mamba_selective_state_amd).

Sizes: the decode layer of this repository's workloads (128 heads x dim 64 = 8192 inner channels, 8 groups, batch
256, speculative batches of 512 x 4 drafts) in a model of width 4096, whose input projection has 2 * 8192 +
2 * 8 * 128 + 128 = 18560 outputs, and generic vocabularies.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_EPS = 1e-5
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _norm(name, rows, dim, dtype, residual=False, gate=False, groups=1, out="same"):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "dtype": dtype, "residual": residual, "gate": gate,
            "groups": groups, "out": out}


def _linear(name, m, n, k, act, dtype, bias=False):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "act": act, "dtype": dtype, "bias": bias}


def _logprob(name, rows, vocab, dtype, top=0, mask=False, temperature=False):
    return {"name": name, "op": "logprob", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "mask": mask,
            "temperature": temperature}


def listed():
    return [
        # the norm before a layer, one sequence: latency
        _norm("norm_one_token", 1, 4096, "bf16", residual=True),
        # the same at the decode batch, with the 8-bit output that the projection takes
        _norm("norm_decode_mxfp8", 256, 4096, "bf16", residual=True, out="mxfp8"),
        # the gated norm after the state update, over a prompt batch
        _norm("norm_gated_prefill_mxfp8", 16384, 8192, "bf16", gate=True, groups=8, out="mxfp8"),
        # a width that no vector access divides, a ragged row count
        _norm("norm_odd", 1237, 2561, "f16", residual=True),
        # the input projection of one sequence: the weights' bytes
        _linear("linear_one_token", 1, 18560, 4096, "mxfp8", "bf16"),
        # the output projection at the decode batch
        _linear("linear_decode", 256, 4096, 8192, "mxfp4", "bf16"),
        # the input projection over a prompt batch: the matrix cores
        _linear("linear_prefill", 8192, 18560, 4096, "mxfp4", "bf16"),
        # ragged everywhere: rows, outputs and an inner size that ends inside every tile
        _linear("linear_odd", 777, 2049, 2592, "mxfp8", "f16", bias=True),
        # one row of logits with alternatives for the answer
        _logprob("logprob_one_row", 1, 65536, "f32", top=5),
        # verification of a speculative batch: 512 sequences x 4 drafts at a temperature
        _logprob("logprob_verify", 2048, 65536, "bf16", temperature=True),
        # constrained decoding: a ragged vocabulary under a mask
        _logprob("logprob_masked", 37, 50021, "f32", top=20, mask=True),
        # scoring with alternatives over a large vocabulary
        _logprob("logprob_score", 1024, 131072, "bf16", top=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "logprob"))
    if op == "norm":
        out = rng.choice(("same", "same", "mxfp8"))
        groups = rng.choice((1, 1, 2, 8))
        unit = groups * (32 if out == "mxfp8" else 1)
        dim = max(unit, _log_int(rng, 64, 16384) // unit * unit)
        rows = _log_int(rng, 1, 16384)
        rows = max(1, min(rows, 16384 * 8192 // dim))
        gate = rng.random() < 0.4
        case = _norm("", rows, dim, rng.choice(("bf16", "f16", "f32")), residual=not gate, gate=gate, groups=groups,
                     out=out)
    elif op == "linear":
        m, n = _log_int(rng, 1, 8192), _log_int(rng, 64, 18560)
        k = _log_int(rng, 256, 8192) // 32 * 32
        m = max(1, min(m, 8192 * 18560 * 4096 // (n * k)))
        case = _linear("", m, n, k, rng.choice(("mxfp8", "mxfp4")), rng.choice(("bf16", "f16")),
                       bias=rng.random() < 0.3)
    else:
        vocab = _log_int(rng, 1000, 131072)
        rows = _log_int(rng, 1, 2048)
        dtype = rng.choice(("bf16", "f16", "f32"))
        rows = max(1, min(rows, 2048 * 65536 * 2 // (vocab * _BYTES[dtype])))
        case = _logprob("", rows, vocab, dtype, top=rng.choice((0, 1, 5, 8, 20)), mask=rng.random() < 0.3,
                        temperature=rng.random() < 0.4)
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "norm":
        dt = _DTYPES[case["dtype"]]
        shape = (case["rows"], case["dim"])
        # hidden states have a few channels far larger than the rest
        channel = torch.where(uniform(case["dim"]) < 0.01, 12.0, 1.0)
        s["x"] = (normal(*shape) * channel).to(dt)
        s["weight"] = (1 + 0.2 * normal(case["dim"])).to(dt)
        s["residual"] = (2 * normal(*shape) * channel).to(dt) if case["residual"] else None
        s["gate"] = normal(*shape).to(dt) if case["gate"] else None
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        channel = torch.where(uniform(k) < 0.01, 8.0, 1.0)
        s["x"] = (normal(m, k) * channel).to(_DTYPES[case["dtype"]])
        # the weights as a checkpoint holds them: codes of two a byte and a scale byte per 32 values
        w = (normal(n, k) / math.sqrt(k)).reshape(n, k // 32, 32)
        e = torch.frexp(w.abs().amax(-1, keepdim=True)).exponent - 3  # floor(log2 amax) - 2
        mag = w.abs() * torch.exp2(-e.float())
        step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
        mag = torch.clamp(torch.round(mag / step) * step, max=6.0)
        code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
        code = torch.where(w < 0, code + 8, code).reshape(n, k)
        s["w"] = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
        s["w_scale"] = (e + 127).to(torch.uint8).reshape(n, k // 32)
        s["bias"] = normal(n) if case["bias"] else None
    else:
        rows, vocab = case["rows"], case["vocab"]
        logits = 2.5 * normal(rows, vocab)
        # a handful of tokens that the model favours, and some that a sampler's rules have ruled out
        part = vocab // 8
        few = torch.randint(0, part, (rows, 8), generator=g, device="cuda") + part * torch.arange(8, device="cuda")
        logits.scatter_(1, few, 9 + 3 * normal(rows, 8))
        logits[uniform(rows, vocab) < 0.002] = -math.inf
        s["mask"] = None
        if case["mask"]:
            words = -(-vocab // 32)
            # a grammar leaves about half of the tokens, and in some rows few
            bits = uniform(rows, words * 32) < torch.where(uniform(rows, 1) < 0.25, 0.001, 0.5)
            weights = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
            packed = (bits.reshape(rows, words, 32) * weights).sum(-1)
            s["mask"] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
        # what was drafted: mostly tokens the model favours too
        any_token = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        s["tokens"] = torch.where(uniform(rows) < 0.7, few[:, 0], any_token)
        s["logits"] = logits.to(_DTYPES[case["dtype"]])
        s["temperature"] = 0.5 + uniform(rows) if case["temperature"] else None
    return s


# ---------------------------------------------------------------- the framework's calls


def _as_floats(codes, scales):
    """MXFP8 bytes as the floating types they are: E4M3 codes and E8M0 (power-of-two) scales."""
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _run_own(s):
    import mamba_selective_state_amd as ssu

    case = s["case"]
    if case["op"] == "norm":
        y = ssu.add_rms_norm(s["x"], s["weight"], residual=s["residual"], gate=s["gate"], groups=case["groups"],
                             eps=_EPS, out_format=None if case["out"] == "same" else case["out"])
        r = {}
        if case["residual"]:
            y, r["residual"] = y
        if case["out"] == "same":
            r["y"] = y
        else:
            r.update(_as_floats(*y))
        return r
    if case["op"] == "linear":
        return {"y": ssu.mx_linear(s["x"], s["w"], s["w_scale"], bias=s["bias"], activation=case["act"])}
    t = ssu.token_logprobs(s["logits"], s["tokens"], top=case["top"], mask=s["mask"], temperature=s["temperature"])
    r = {"logprob": t.logprob, "entropy": t.entropy, "rank": t.rank}
    if case["top"]:
        r.update(top_tokens=t.top_tokens, top_logprobs=t.top_logprobs)
    return r


# ---------------------------------------------------------------- the plain forms


def _block_scale(x, emax):
    """The power-of-two scale of each block of 32: floor(log2 max|x|) - emax, and x over it."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - emax, -126).clamp(-126, 127)
    return torch.ldexp(torch.ones_like(amax), e), torch.ldexp(b, -e)


def _round_e4m3(v):
    e = (torch.frexp(v).exponent - 1).clamp(min=-6) - 3
    return torch.ldexp(torch.round(torch.ldexp(v, -e)), e).clamp(-448, 448)


def _round_e2m1(v):
    e = (torch.frexp(v).exponent - 1).clamp(min=0) - 1
    return torch.ldexp(torch.round(torch.ldexp(v, -e)), e).clamp(-6, 6)


def _plain_norm(s):
    case = s["case"]
    u = s["x"].float()
    r = {}
    if case["gate"]:
        z = s["gate"].float()
        u = u * (z / (1 + torch.exp(-z)))
    if case["residual"]:
        u = u + s["residual"].float()
        r["residual"] = u.to(s["x"].dtype)
    part = u.reshape(u.shape[0], case["groups"], -1)
    part = part * torch.rsqrt((part * part).mean(-1, keepdim=True) + _EPS)
    y = part.reshape(u.shape) * s["weight"].float()
    if case["out"] == "same":
        r["y"] = y.to(s["x"].dtype)
    else:
        scale, v = _block_scale(y, 8)
        r["codes"] = _round_e4m3(v).reshape(y.shape).to(torch.float8_e4m3fn)
        r["scales"] = scale[..., 0].to(torch.float8_e8m0fnu)
    return r


def _decode_weights(w, w_scale, dtype):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=w.device, dtype=dtype)
    codes = torch.stack((w & 15, w >> 4), -1).reshape(w.shape[0], -1, 32)
    scale = torch.exp2(w_scale.to(dtype) - 127)
    return (table[codes.long()] * scale[..., None]).reshape(w.shape[0], -1)


def _plain_linear(s):
    case = s["case"]
    scale, v = _block_scale(s["x"].float(), 8 if case["act"] == "mxfp8" else 2)
    v = _round_e4m3(v) if case["act"] == "mxfp8" else _round_e2m1(v)
    a = (v * scale).reshape(s["x"].shape)
    y = a @ _decode_weights(s["w"], s["w_scale"], torch.float32).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype)}


def _allowed(s):
    """Which tokens of each row count: allowed by the mask, and with a logit above -inf."""
    ok = s["logits"] > -math.inf
    if s["mask"] is not None:
        at = torch.arange(ok.shape[1], device=ok.device)
        ok &= ((s["mask"][:, at // 32] >> (at % 32)) & 1) == 1
    return ok


def _plain_logprob(s):
    case = s["case"]
    ok = _allowed(s)
    raw = torch.where(ok, s["logits"].float(), -math.inf)
    x = raw if s["temperature"] is None else raw / s["temperature"][:, None]
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    total = torch.exp(x - top).sum(-1, keepdim=True)
    logp = torch.where(ok, x - top - torch.log(total), -math.inf)
    r = {"entropy": -torch.where(ok, torch.exp(logp) * logp, 0.0).sum(-1)}
    token = s["tokens"][:, None]
    r["logprob"] = logp.gather(1, token)[:, 0]
    mine = raw.gather(1, token)
    at = torch.arange(raw.shape[1], device=raw.device)
    before = ((raw > mine) | ((raw == mine) & (at < token))).sum(-1)
    r["rank"] = torch.where(ok.gather(1, token)[:, 0], before, -1).to(torch.int32)
    if case["top"]:
        first = torch.sort(raw, dim=-1, descending=True, stable=True)
        best, ids = first.values[:, :case["top"]], first.indices[:, :case["top"]]
        r["top_tokens"] = torch.where(best > -math.inf, ids, -1).to(torch.int32)
        r["top_logprobs"] = logp.gather(1, ids)
    return r


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "linear": _plain_linear, "logprob": _plain_logprob}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "norm":
        n, b = case["rows"] * case["dim"], _BYTES[case["dtype"]]
        moved = n * b * (1 + 2 * case["residual"] + case["gate"]) + case["dim"] * b
        moved += n * b if case["out"] == "same" else n + n // 32
        return {"bytes": moved, "flops": n * (4 + case["residual"] + 4 * case["gate"])}
    if case["op"] == "linear":
        m, n, k, b = case["m"], case["n"], case["k"], _BYTES[case["dtype"]]
        return {"bytes": m * k * b + n * k // 2 + n * k // 32 + m * n * b + 4 * n * case["bias"], "flops": 2 * m * n * k}
    n = case["rows"] * case["vocab"]
    moved = n * _BYTES[case["dtype"]] + (n // 8 if case["mask"] else 0)
    return {"bytes": moved + case["rows"] * (20 + 8 * case["top"] + 4 * case["temperature"]), "flops": 6 * n}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_blocks(y, largest, values):
    """Each block's scale, the largest power of two X with `largest` * X <= max|y| (`largest`: the format's top power
    of two), and every value over it taken to the nearest of `values`, the even one of two as near."""
    b = y.reshape(*y.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    k = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    k = torch.where(torch.exp2(k) > amax, k - 1, k)
    k = torch.where(torch.exp2(k + 1) <= amax, k + 1, k)
    scale = torch.exp2(torch.where(amax > 0, k - math.log2(largest), -126.0).clamp(-126, 127))
    v = (b / scale).contiguous()
    grid = torch.tensor(values, dtype=y.dtype, device=y.device)
    hi = torch.searchsorted(grid, v.abs().contiguous()).clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - v.abs(), v.abs() - grid[lo]
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return scale, torch.sign(v) * grid[pick]


def _e4m3_values():
    """The finite magnitudes of E4M3 in order of their codes (so an even place is an even code)."""
    sub = [m / 8 * 2.0 ** -6 for m in range(8)]
    return sub + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        u = s["x"].double()
        r = {}
        if case["gate"]:
            u = u * s["gate"].double() * torch.sigmoid(s["gate"].double())
        if case["residual"]:
            u = u + s["residual"].double()
            r["residual"] = u
        chunks = u.unflatten(-1, (case["groups"], -1))
        y = (chunks / torch.sqrt(chunks.pow(2).mean(-1, keepdim=True) + _EPS)).flatten(-2) * s["weight"].double()
        if case["out"] == "same":
            r["y"] = y
        else:
            scale = _exact_blocks(y, 256.0, _e4m3_values())[0]
            # the codes before their rounding, as for any other output
            r["codes"], r["scales"] = (y.unflatten(-1, (-1, 32)) / scale).flatten(-2), scale[..., 0]
        return r
    if case["op"] == "linear":
        form = (256.0, _e4m3_values()) if case["act"] == "mxfp8" else (4.0, list(_E2M1))
        scale, v = _exact_blocks(s["x"].double(), *form)
        a = (v * scale).flatten(-2)
        grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
        low, high = s["w"].long() % 16, s["w"].long() // 16
        w = torch.empty(case["n"], case["k"], dtype=torch.float64, device="cuda")
        for at, c in ((0, low), (1, high)):
            w[:, at::2] = grid[c % 8] * (1.0 - 2.0 * (c // 8))
        w = w * torch.pow(2.0, s["w_scale"].double() - 127).repeat_interleave(32, -1)
        y = torch.mm(a, w.t())
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    l = s["logits"].double()
    ok = ~torch.isneginf(l)
    if case["mask"]:
        bits = (s["mask"].long() & 0xFFFFFFFF)[..., None] // (2 ** torch.arange(32, device="cuda")) % 2
        ok = ok & bits.flatten(-2)[:, :case["vocab"]].bool()
    if case["temperature"]:
        l = l / s["temperature"].double()[:, None]
    l = l.masked_fill(~ok, -math.inf)
    some = ok.any(-1)
    lse = torch.where(some, torch.logsumexp(l, -1), 0.0)
    p = torch.where(ok, torch.exp(l - lse[:, None]), 0.0)
    entropy = torch.where(some, lse - (p * l.masked_fill(~ok, 0.0)).sum(-1), 0.0)
    r = {"entropy": entropy, "logprob": (l - lse[:, None]).gather(1, s["tokens"][:, None])[:, 0], "rank": None}
    if case["top"]:
        best = torch.topk(l, case["top"], -1).values
        r.update(top_tokens=None, top_logprobs=best - lse[:, None])
    return r
