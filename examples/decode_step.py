#!/usr/bin/env python3
"""A speculative decode step of a small Mamba-2 model with random weights, run by this
framework's operators end to end:

    per layer   h, r = add_rms_norm(x, w, residual)      MXFP8 codes and scales
                z, x, B, C, dt = mx_linear(h, W_in)      MXFP4 weights
                y = selective_state_update(...)          T draft tokens per sequence
                g = add_rms_norm(y, w, gate=z, groups)   MXFP8 codes and scales
                x = mx_linear(g, W_out)
    at the end  logits = mx_linear(add_rms_norm(x, w, residual), W_head)
                token_logprobs(logits, the next drafts): what a verifier accepts by,
                and the alternatives to answer with

    python examples/decode_step.py [--batch 8] [--drafts 3] [--layers 4] [--check]

The convolution over x, B and C, which comes before the state update in the full model, is
left out. --check runs the same step in plain torch from the same codes and prints the
largest difference of a log probability.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_selective_state_amd as ssu  # noqa: E402

EPS = 1e-5


def make_model(layers, width, heads, dim, dstate, groups, vocab, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    inner = heads * dim

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def weight(n, k):
        return ssu.mx_quantize(normal(n, k) / math.sqrt(k), "mxfp4")
    model = {"sizes": (width, heads, dim, dstate, groups, vocab), "layers": []}
    for _ in range(layers):
        model["layers"].append({
            "norm": (1 + 0.1 * normal(width)).bfloat16(),
            "in": weight(2 * inner + 2 * groups * dstate + heads, width),
            "A": -torch.exp(torch.rand(heads, generator=g, device="cuda") * 2), "D": normal(heads),
            "dt_bias": normal(heads) - 3,
            "gated_norm": (1 + 0.1 * normal(inner)).bfloat16(),
            "out": weight(width, inner)})
    model["norm"] = (1 + 0.1 * normal(width)).bfloat16()
    model["head"] = weight(vocab, width)
    model["embedding"] = normal(vocab, width).bfloat16()
    return model


def split(zxbcdt, sizes, batch, drafts):
    """The input projection's outputs as z, x, B, C and dt of [batch, drafts, ...] views."""
    width, heads, dim, dstate, groups, _ = sizes
    inner, gn = heads * dim, groups * dstate
    z, x, B, C, dt = torch.split(zxbcdt, [inner, inner, gn, gn, heads], dim=-1)

    def rows(t, *shape):
        return t.unflatten(0, (batch, drafts)).unflatten(-1, shape)
    return z, rows(x, heads, dim), rows(B, groups, dstate), rows(C, groups, dstate), dt.unflatten(0, (batch, drafts))


def step(model, states, tokens, next_tokens, top=3):
    """One step of `tokens` [batch, drafts]: every layer's state (read at the slot of the
    sequence, one snapshot slot written per draft) moves on. Returns TokenLogprobs of
    `next_tokens` and the logits."""
    sizes = model["sizes"]
    heads, dim = sizes[1], sizes[2]
    batch, drafts = tokens.shape
    read = torch.arange(batch, device="cuda", dtype=torch.int32)[:, None].expand(batch, drafts)
    write = batch + torch.arange(batch * drafts, device="cuda", dtype=torch.int32).view(batch, drafts)
    x = model["embedding"][tokens.flatten()]
    residual = torch.zeros(x.shape, dtype=torch.float32, device="cuda")
    for layer, state in zip(model["layers"], states):
        h, residual = ssu.add_rms_norm(x, layer["norm"], residual, eps=EPS, out_format="mxfp8",
                                       residual_out=residual)
        z, xs, B, C, dt = split(ssu.mx_linear(h, *layer["in"]), sizes, batch, drafts)
        y = ssu.selective_state_update(state, xs, dt, layer["A"], B, C, layer["D"], dt_bias=layer["dt_bias"],
                                       dt_softplus=True, state_batch_indices=read, dst_state_batch_indices=write)
        g = ssu.add_rms_norm(y.view(batch * drafts, heads * dim), layer["gated_norm"], gate=z, groups=sizes[4],
                             eps=EPS, out_format="mxfp8")
        x = ssu.mx_linear(g, *layer["out"])
    h, _ = ssu.add_rms_norm(x, model["norm"], residual, eps=EPS, out_format="mxfp8")
    logits = ssu.mx_linear(h, *model["head"], out_dtype=torch.float32)
    return ssu.token_logprobs(logits, next_tokens.flatten(), top=top), logits


# ---------------------------------------------------------------- the same in plain torch


def decode(codes, scales):
    """float32 values of MXFP8 (as many codes as 32 times the scales) or MXFP4 codes."""
    if codes.shape[-1] == 32 * scales.shape[-1]:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
        table = torch.cat((e2m1, -e2m1))
        v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    return v * torch.exp2(scales.float() - 127).repeat_interleave(32, -1)


def plain_norm(u, weight, groups=1):
    p = u.unflatten(-1, (groups, -1))
    p = p * torch.rsqrt(p.square().mean(-1, keepdim=True) + EPS)
    return decode(*ssu.mx_quantize((p.flatten(-2) * weight.float()).contiguous(), "mxfp8"))


def plain_step(model, states, tokens, next_tokens):
    sizes = model["sizes"]
    width, heads, dim, dstate, groups, _ = sizes
    batch, drafts = tokens.shape
    x = model["embedding"][tokens.flatten()]
    residual = torch.zeros(x.shape, dtype=torch.float32, device="cuda")
    for layer, state in zip(model["layers"], states):
        residual = residual + x.float()
        zxbcdt = (plain_norm(residual, layer["norm"]) @ decode(*layer["in"]).t()).bfloat16()
        z, xs, B, C, dt = (t.float() for t in split(zxbcdt, sizes, batch, drafts))
        dt = torch.nn.functional.softplus(dt + layer["dt_bias"])
        s, ys = state[:batch].clone(), []
        for t in range(drafts):
            Bh = B[:, t].repeat_interleave(heads // groups, 1)
            Ch = C[:, t].repeat_interleave(heads // groups, 1)
            s = s * torch.exp(dt[:, t] * layer["A"])[..., None, None] + (dt[:, t, :, None] * xs[:, t])[..., None] * Bh[:, :, None]
            ys.append((s * Ch[:, :, None]).sum(-1) + layer["D"][:, None] * xs[:, t])
        y = torch.stack(ys, 1).bfloat16().float().view(batch * drafts, heads * dim)
        g = plain_norm(y * torch.nn.functional.silu(z), layer["gated_norm"], groups)
        x = (g @ decode(*layer["out"]).t()).bfloat16()
    logits = plain_norm(residual + x.float(), model["norm"]) @ decode(*model["head"]).t()
    return torch.log_softmax(logits, -1).gather(1, next_tokens.flatten()[:, None])[:, 0], logits


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--vocab", type=int, default=4099)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    dim, dstate, groups = 64, 128, 2
    model = make_model(a.layers, a.width, a.heads, dim, dstate, groups, a.vocab)
    g = torch.Generator(device="cuda").manual_seed(1)
    slots = a.batch * (1 + a.drafts)
    states = [0.1 * torch.randn((slots, a.heads, dim, dstate), generator=g, device="cuda") for _ in range(a.layers)]
    tokens = torch.randint(0, a.vocab, (a.batch, a.drafts + 1), generator=g, device="cuda")
    before = [s.clone() for s in states]
    r, logits = step(model, states, tokens[:, :-1], tokens[:, 1:])
    print("log probabilities of the drafts, first sequence:", [round(v, 3) for v in r.logprob[:a.drafts].tolist()])
    print("their ranks:", r.rank[:a.drafts].tolist(), " entropies:", [round(v, 3) for v in r.entropy[:a.drafts].tolist()])
    print("alternatives to the first:", list(zip(r.top_tokens[0].tolist(), [round(v, 3) for v in r.top_logprobs[0].tolist()])))
    if not a.check:
        return None
    want, plain_logits = plain_step(model, before, tokens[:, :-1], tokens[:, 1:])
    off = float((r.logprob - want).abs().max())
    print("largest difference to plain torch: log probability %.4f, logit %.4f of %.2f"
          % (off, float((logits - plain_logits).abs().max()), float(plain_logits.abs().max())))
    return off


if __name__ == "__main__":
    main()
