"""The cases by which the operators of a beam search over many requests are measured: beam_select and
reorder_states (the choice of continuations, and the sequence states that follow it) and add_lora (low-rank
adapters of many requests beside a shared projection), of mamba_selective_state_amd.

Sizes: the decode layer of this repository's workloads (128 heads x dim 64 = 8192 inner channels, 8 groups,
dstate 128, batch 256, speculative batches of 512 x 4 drafts) in a model of width 4096, whose input projection
has 2 * 8192 + 2 * 8 * 128 + 128 = 18560 outputs and whose convolution keeps 3 tokens of 8192 + 2 * 8 * 128 =
10240 channels; and generic vocabularies, beams and ranks.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_END = 2  # the token that ends a sequence


def _beam(name, batch, beams, vocab, keep, dtype, mask=False, ended=False):
    return {"name": name, "op": "beam", "batch": batch, "beams": beams, "vocab": vocab, "keep": keep, "dtype": dtype,
            "mask": mask, "ended": ended}


def _reorder(name, batch, beams, layers, heads, dim, dstate, channels, dtype, short=False):
    return {"name": name, "op": "reorder", "batch": batch, "beams": beams, "layers": layers, "heads": heads,
            "dim": dim, "dstate": dstate, "channels": channels, "dtype": dtype, "short": short}


def _lora(name, rows, k, n, rank, loaded, used, dtype, order, x="same", some=False):
    return {"name": name, "op": "lora", "rows": rows, "k": k, "n": n, "rank": rank, "loaded": loaded, "used": used,
            "dtype": dtype, "order": order, "x": x, "some": some}


def listed():
    return [
        # one request's step: latency
        _beam("beam_one", 1, 4, 65536, 8, "f32"),
        # a decode batch; twice as many continuations as beams, since some of them end
        _beam("beam_decode", 32, 8, 65536, 16, "bf16"),
        # constrained decoding over a ragged vocabulary, some beams already ended or not yet begun
        _beam("beam_masked", 37, 5, 50021, 10, "f32", mask=True, ended=True),
        # the largest: every sequence of a batch of 256 searched with 8 beams over a large vocabulary
        _beam("beam_large", 256, 8, 131072, 16, "bf16", ended=True),
        # one request, one layer's state and convolution: latency
        _reorder("reorder_one", 1, 4, 1, 128, 64, 128, 10240, "f32"),
        # a batch of 8 requests x 8 beams, eight layers with their convolutions
        _reorder("reorder_layers", 8, 8, 8, 128, 64, 128, 10240, "bf16"),
        # slots whose sizes no vector access divides, and beams that the search has left empty
        _reorder("reorder_odd", 37, 5, 3, 3, 17, 13, 205, "f32", short=True),
        # one token of one request: latency
        _lora("lora_one_token", 1, 4096, 18560, 16, 32, 1, "bf16", "mixed"),
        # the output projection at the decode batch, every row another request's
        _lora("lora_decode", 256, 8192, 4096, 16, 64, 48, "bf16", "mixed"),
        # the input projection of a speculative batch, on the 8-bit rows that the norm before it gives
        _lora("lora_drafts_mxfp8", 2048, 4096, 18560, 16, 64, 64, "bf16", "runs", x="mxfp8"),
        # the same over a prompt batch of a few requests
        _lora("lora_prefill", 8192, 4096, 18560, 64, 16, 8, "bf16", "runs"),
        # ragged everywhere, rows without an adapter among them
        _lora("lora_odd", 777, 2592, 2049, 20, 13, 11, "f16", "mixed", some=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("beam", "reorder", "lora"))
    if op == "beam":
        vocab, beams = _log_int(rng, 1000, 131072), _log_int(rng, 1, 24)
        dtype = rng.choice(("bf16", "f16", "f32"))
        batch = max(1, min(_log_int(rng, 1, 256), 2048 * 131072 * 2 // (beams * vocab * _BYTES[dtype])))
        keep = min(32, beams * rng.choice((1, 2)))
        case = _beam("", batch, beams, vocab, keep, dtype, mask=rng.random() < 0.3, ended=rng.random() < 0.5)
    elif op == "reorder":
        heads, dim, dstate = _log_int(rng, 1, 128), _log_int(rng, 8, 128), rng.choice((16, 64, 128, 13, 100))
        dtype, beams = rng.choice(("bf16", "f16", "f32")), _log_int(rng, 1, 24)
        channels = heads * dim + rng.choice((0, 16, 2 * dstate, 2 * 8 * dstate))
        slot = (heads * dim * dstate + 3 * channels) * _BYTES[dtype]
        layers = rng.choice((1, 1, 2, 4, 8))
        most = 64 * 8 * 128 * 64 * 128 * 2  # bytes of the largest listed pools
        while layers * beams * slot > most:
            layers, beams = max(1, layers // 2), max(1, beams // 2)
        batch = max(1, min(_log_int(rng, 1, 64), most // (layers * beams * slot)))
        case = _reorder("", batch, beams, layers, heads, dim, dstate, channels, dtype, short=rng.random() < 0.3)
    else:
        x = rng.choice(("same", "same", "same", "mxfp8", "mxfp4"))
        dtype = "bf16" if x != "same" else rng.choice(("bf16", "bf16", "f16", "f32"))
        unit = 1 if x == "same" else 32
        k, n = max(unit, _log_int(rng, 64, 8192) // unit * unit), _log_int(rng, 64, 18560)
        rank = rng.choice((4, 8, 16, 16, 32, 64, 128, 20))
        loaded = min(_log_int(rng, 1, 64), 1024 // rank)
        rows = _log_int(rng, 1, 8192)
        rows = max(1, min(rows, 8192 * (4096 + 2 * 18560) * 2 // ((k + 2 * n) * _BYTES[dtype])))
        some = rng.random() < 0.3
        used = min(rng.randint(1, loaded), _with_adapter(rows, some))
        case = _lora("", rows, k, n, rank, loaded, used, dtype, rng.choice(("mixed", "runs")), x=x, some=some)
    del case["name"]
    return case


def _ended(b, i):
    return (b + 2 * i) % 7 == 3


def _begun(b, i):
    return i == 0 or (b + i) % 11 != 5


def _with_adapter(rows, some):
    return rows - rows // 5 if some else rows


def _survivors(case):
    """How many beams of a request have a successor, and how many successors there are."""
    beams = case["beams"]
    return max(1, round(0.6 * beams)), max(1, beams - 1) if case["short"] else beams


# ---------------------------------------------------------------- inputs


def _block_scale(x, emax):
    """The power-of-two scale of each block of 32: floor(log2 max|x|) - emax, and x over it."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - emax, -126).clamp(-126, 127)
    return e, torch.ldexp(b, -e)


def _quantized(x, form):
    """The codes and scale bytes of rows in MXFP8 or MXFP4, as the norm before a projection gives them."""
    e, v = _block_scale(x, 8 if form == "mxfp8" else 2)
    scales = (e + 127).to(torch.uint8)[..., 0]
    if form == "mxfp8":
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape), scales
    mag = v.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    mag = torch.clamp(torch.round(mag / step) * step, max=6.0)
    code = torch.where(mag < 2, mag * 2, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
    code = torch.where(v < 0, code + 8, code).reshape(x.shape)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "beam":
        batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
        rows = batch * beams
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
        s["logits"] = logits.to(_DTYPES[case["dtype"]])
        # log probabilities of the sequences so far, best first
        s["scores"] = -20 * uniform(batch, 1) - 4 * torch.sort(uniform(batch, beams), -1).values
        s["finished"] = None
        if case["ended"]:
            b, i = torch.arange(batch, device="cuda")[:, None], torch.arange(beams, device="cuda")
            s["finished"] = ((b + 2 * i) % 7 == 3)
            s["scores"] = torch.where((i == 0) | ((b + i) % 11 != 5), s["scores"], -math.inf)
    elif case["op"] == "reorder":
        batch, beams, dt = case["batch"], case["beams"], _DTYPES[case["dtype"]]
        survivors, kept = _survivors(case)
        survivors = min(survivors, kept)
        slots = batch * beams + 3  # a pool has slots of other sequences too
        s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:batch * beams].reshape(batch, beams).to(torch.int32)
        alive = torch.argsort(uniform(batch, beams), -1)[:, :survivors]
        again = torch.randint(0, survivors, (batch, kept - survivors), generator=g, device="cuda")
        parents = torch.cat((alive, alive.gather(1, again)), 1)
        parents = parents.gather(1, torch.argsort(uniform(batch, kept), -1))
        s["parents"] = torch.nn.functional.pad(parents, (0, beams - kept), value=-1).to(torch.int32)
        s["pools"] = []
        for _ in range(case["layers"]):
            s["pools"].append(torch.randn((slots, case["heads"], case["dim"], case["dstate"]), generator=g, device="cuda", dtype=dt))
            s["pools"].append(torch.randn((slots, case["channels"], 3), generator=g, device="cuda", dtype=dt))
    else:
        rows, k, n, rank, loaded = case["rows"], case["k"], case["n"], case["rank"], case["loaded"]
        dt = _DTYPES[case["dtype"]]
        # hidden states have a few channels larger than the rest
        x = normal(rows, k) * torch.where(uniform(k) < 0.01, 8.0, 1.0)
        s["x"] = x.to(dt) if case["x"] == "same" else _quantized(x, case["x"])
        s["a"] = (normal(loaded, rank, k) / math.sqrt(k)).to(dt)
        s["b"] = (0.3 * normal(loaded, n, rank)).to(dt)
        s["scale"] = 0.5 + uniform(loaded)
        s["y"] = normal(rows, n).to(dt)  # the shared projection's outputs
        # `used` of the adapters, each at least once
        with_one = _with_adapter(rows, case["some"])
        some = torch.randperm(loaded, generator=g, device="cuda")[:case["used"]]
        ids = some[torch.cat((torch.arange(case["used"], device="cuda"),
                              torch.randint(0, case["used"], (with_one - case["used"],), generator=g, device="cuda")))]
        if case["order"] == "mixed":
            ids = ids[torch.randperm(with_one, generator=g, device="cuda")]
        else:  # a request's tokens follow each other
            ids = torch.sort(ids).values
        if case["some"]:
            at = torch.arange(rows, device="cuda")
            ids = torch.where(at % 5 == 4, -1, ids[(at - at // 5).clamp(max=with_one - 1)])
        s["ids"] = ids.to(torch.int32)
    return s


# ---------------------------------------------------------------- the framework's calls


def _run_own(s):
    import mamba_selective_state_amd as ssu

    case = s["case"]
    if case["op"] == "beam":
        r = ssu.beam_select(s["logits"], s["scores"], case["keep"], finished=s["finished"], end_token=_END, mask=s["mask"])
        return {"scores": r.scores, "parents": r.parents, "tokens": r.tokens}
    if case["op"] == "reorder":
        return {"slots": ssu.reorder_states(s["pools"], s["slots"], s["parents"]), "pools": s["pools"]}
    return {"y": ssu.add_lora(s["y"], s["x"], s["a"], s["b"], s["ids"], scale=s["scale"])}


# ---------------------------------------------------------------- the plain forms


def _allowed(s):
    """Which tokens of each row count: allowed by the mask, and with a logit above -inf."""
    ok = s["logits"] > -math.inf
    if s["mask"] is not None:
        at = torch.arange(ok.shape[1], device=ok.device)
        ok &= ((s["mask"][:, at // 32] >> (at % 32)) & 1) == 1
    return ok


def _plain_beam(s):
    case = s["case"]
    batch, beams, keep = case["batch"], case["beams"], case["keep"]
    raw = torch.where(_allowed(s), s["logits"].float(), -math.inf)
    top = raw.amax(-1)
    top = torch.where(top > -math.inf, top, 0.0)
    # in 64 bits: scores of two beams that are near each other decide which of them goes on
    lse = top.double() + torch.log(torch.exp(raw - top[:, None]).sum(-1, dtype=torch.float64))
    first = torch.sort(raw, dim=-1, descending=True, stable=True)
    best, ids = (t[:, :keep].reshape(batch, beams, keep) for t in (first.values, first.indices))
    score = s["scores"].double()[..., None]
    c = torch.where(best > -math.inf, score + (best.double() - lse.reshape(batch, beams, 1)), -math.inf)
    if s["finished"] is not None:
        place = torch.arange(keep, device=c.device)
        c = torch.where(s["finished"][..., None], torch.where(place == 0, score, -math.inf), c)
        ids = torch.where(s["finished"][..., None], _END, ids)
    chosen = torch.sort(c.reshape(batch, beams * keep), dim=-1, descending=True, stable=True)
    c, at = chosen.values[:, :keep], chosen.indices[:, :keep]
    return {"scores": c.float(), "parents": torch.where(c > -math.inf, at // keep, -1).to(torch.int32),
            "tokens": torch.where(c > -math.inf, ids.reshape(batch, beams * keep).gather(1, at), -1).to(torch.int32)}


def _plain_reorder(s):
    slots, p = s["slots"].long(), s["parents"].long()
    beams = slots.shape[1]
    at = torch.arange(beams, device=p.device)
    first = (p >= 0) & ~((p[:, :, None] == p[:, None, :]) & (at[:, None] > at)).any(-1)
    used = (p[:, :, None] == at).any(1)
    free = torch.argsort(used.to(torch.int32), dim=-1, stable=True)  # beams without a successor first
    place = (torch.cumsum((~first).to(torch.int64), -1) - 1).clamp(min=0)
    source = slots.gather(1, p.clamp(min=0))
    new = torch.where(first, source, slots.gather(1, free.gather(1, place)))
    copied = (p >= 0) & ~first
    src, dst = source[copied], new[copied]
    for pool in s["pools"]:
        pool[dst] = pool[src]
    return {"slots": new.to(torch.int32), "pools": s["pools"]}


def _floats(x):
    """The rows that a projection takes, in 32 bits."""
    if isinstance(x, torch.Tensor):
        return x.float()
    codes, scales = x
    if codes.shape[-1] == 32 * scales.shape[-1]:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
        v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    return v * torch.exp2(scales.float() - 127).repeat_interleave(32, -1)


def _plain_lora(s):
    a, b = s["a"].float(), s["b"].float()
    h = (_floats(s["x"]) @ a.flatten(0, 1).t()).unflatten(1, a.shape[:2])
    mine = s["ids"][:, None] == torch.arange(a.shape[0], device=a.device)
    h = torch.where(mine[..., None], h * s["scale"][:, None], 0.0)
    y = s["y"].float() + h.flatten(1) @ b.transpose(1, 2).flatten(0, 1)
    s["y"].copy_(torch.where((s["ids"] >= 0)[:, None], y.to(s["y"].dtype), s["y"]))
    return {"y": s["y"]}


def run(state):
    if own:
        return _run_own(state)
    return {"beam": _plain_beam, "reorder": _plain_reorder, "lora": _plain_lora}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    if case["op"] == "beam":
        batch, beams = case["batch"], case["beams"]
        live = batch * beams
        if case["ended"]:
            live = sum(_begun(b, i) and not _ended(b, i) for b in range(batch) for i in range(beams))
        n = live * case["vocab"]
        moved = n * _BYTES[case["dtype"]] + (n // 8 if case["mask"] else 0)
        return {"bytes": moved + batch * (5 * beams + 12 * case["keep"]), "flops": 4 * n}
    if case["op"] == "reorder":
        survivors, kept = _survivors(case)
        copies = case["batch"] * max(0, kept - survivors)
        slot = (case["heads"] * case["dim"] * case["dstate"] + 3 * case["channels"]) * _BYTES[case["dtype"]]
        return {"bytes": 2 * copies * case["layers"] * slot + 12 * case["batch"] * case["beams"], "flops": 0}
    rows, k, n, rank, b = _with_adapter(case["rows"], case["some"]), case["k"], case["n"], case["rank"], _BYTES[case["dtype"]]
    x = {"same": k * b, "mxfp8": k + k // 32, "mxfp4": k // 2 + k // 32}[case["x"]]
    return {"bytes": rows * (x + 2 * n * b) + case["used"] * (rank * (k + n) * b + 4) + 4 * case["rows"],
            "flops": 2 * rows * rank * (k + n)}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "beam":
        l = s["logits"].double()
        ok = ~torch.isneginf(l)
        if case["mask"]:
            bits = (s["mask"].long() & 0xFFFFFFFF)[..., None] // (2 ** torch.arange(32, device="cuda")) % 2
            ok = ok & bits.flatten(-2)[:, :case["vocab"]].bool()
        l = l.masked_fill(~ok, -math.inf)
        best = torch.topk(l, case["keep"], -1).values - torch.logsumexp(l, -1, keepdim=True)
        best = torch.where(torch.isnan(best), -math.inf, best).reshape(case["batch"], case["beams"], case["keep"])
        score = s["scores"].double()[..., None]
        c = score + best
        if case["ended"]:
            c = c.masked_fill(s["finished"][..., None], -math.inf)
            c[..., :1] = torch.where(s["finished"][..., None], score, c[..., :1])
        return {"scores": torch.topk(c.flatten(1), case["keep"], -1).values, "parents": None, "tokens": None}
    if case["op"] == "reorder":
        before = [p.clone() for p in s["pools"]]
        for mine, parents in zip(s["slots"].tolist(), s["parents"].tolist()):
            free = [slot for i, slot in enumerate(mine) if i not in parents]
            taken = set()
            for p in parents:
                if p in taken or p < 0:
                    to = free.pop(0)
                    if p >= 0:
                        for pool, old in zip(s["pools"], before):
                            pool[to] = old[mine[p]]
                taken.add(p)
        return {"slots": None, "pools": [p.double() for p in s["pools"]]}
    y = s["y"].double()
    if case["x"] == "same":
        x = s["x"].double()
    else:
        codes, scales = (t.long() for t in s["x"])
        if case["x"] == "mxfp8":
            e, m = codes // 8 % 16, (codes % 8).double()
            v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6) * (1 - 2 * (codes // 128))
        else:
            grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
            v = torch.empty(case["rows"], case["k"], dtype=torch.float64, device="cuda")
            for at, c in ((0, codes % 16), (1, codes // 16)):
                v[:, at::2] = grid[c % 8] * (1 - 2 * (c // 8))
        x = v * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)
    for i in range(case["loaded"]):
        rows = torch.nonzero(s["ids"] == i)[:, 0]
        if len(rows):
            h = torch.mm(x[rows], s["a"][i].double().t())
            y[rows] += s["scale"][i].double() * torch.mm(h, s["b"][i].double().t())
    return {"y": y}
