#!/usr/bin/env python3
"""Beam search over several requests with a small Mamba-2 model with random weights, every request with a
low-rank adapter of its own beside the shared projections:

    per layer   h, r = add_rms_norm(x, w, residual)      MXFP8 codes and scales
                v = mx_linear(h, W_in); add_lora(v, h, A_in, B_in, adapter)
                y = selective_state_update(...)          one token a beam, in the beam's slot
                g = add_rms_norm(y, w, gate=z, groups)
                x = mx_linear(g, W_out); add_lora(x, g, A_out, B_out, adapter)
    at the end  logits = mx_linear(add_rms_norm(x, w, residual), W_head)
                scores, parents, tokens = beam_select(logits, scores, beams, finished, end)
                slots = reorder_states(states, slots, parents)

    python examples/beam_search.py [--requests 4] [--beams 5] [--steps 8] [--check]

--check runs the best sequences again one token after another in plain torch, with states of their own, and
prints the largest difference of a score.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_selective_state_amd as ssu  # noqa: E402
from examples.decode_step import EPS, decode, make_model, plain_norm, split  # noqa: E402

START, END = 1, 2


def make_adapters(model, count, rank, seed=3):
    """Adapters of every layer's two projections, and their scales. Nobody uses the last one."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width, heads, dim = model["sizes"][:3]
    inner = heads * dim

    def pair(n, k):
        return [(torch.randn(shape, generator=g, device="cuda") * f).bfloat16()
                for shape, f in (((count, rank, k), k ** -0.5), ((count, n, rank), 0.3))]
    layers = [{"in": pair(layer["in"][0].shape[0], width), "out": pair(width, inner)} for layer in model["layers"]]
    return {"layers": layers, "scale": 0.5 + torch.rand(count, generator=g, device="cuda")}


def step(model, adapters, states, slots, tokens, adapter):
    """Logits [batch, beams, vocab] of the tokens [batch, beams]; the states at `slots` move on. `adapter`: one for
    each request, -1 for none."""
    sizes = model["sizes"]
    heads, dim, groups, vocab = sizes[1], sizes[2], sizes[4], sizes[5]
    rows = tokens.numel()
    ids = adapter[:, None].expand(tokens.shape).reshape(rows)
    at = slots.flatten()
    x = model["embedding"][tokens.flatten()]
    residual = torch.zeros(x.shape, dtype=torch.float32, device="cuda")
    for layer, low, state in zip(model["layers"], adapters["layers"], states):
        h, residual = ssu.add_rms_norm(x, layer["norm"], residual, eps=EPS, out_format="mxfp8", residual_out=residual)
        v = ssu.add_lora(ssu.mx_linear(h, *layer["in"]), h, *low["in"], ids, scale=adapters["scale"])
        z, xs, B, C, dt = split(v, sizes, rows, 1)
        y = ssu.selective_state_update(state, xs[:, 0], dt[:, 0], layer["A"], B[:, 0], C[:, 0], layer["D"],
                                       dt_bias=layer["dt_bias"], dt_softplus=True, state_batch_indices=at,
                                       dst_state_batch_indices=at)
        g = ssu.add_rms_norm(y.reshape(rows, heads * dim), layer["gated_norm"], gate=z, groups=groups, eps=EPS,
                             out_format="mxfp8")
        x = ssu.add_lora(ssu.mx_linear(g, *layer["out"]), g, *low["out"], ids, scale=adapters["scale"])
    h, _ = ssu.add_rms_norm(x, model["norm"], residual, eps=EPS, out_format="mxfp8")
    return ssu.mx_linear(h, *model["head"], out_dtype=torch.float32).view(*tokens.shape, vocab)


def search(model, adapters, adapter, beams, steps):
    """The best `beams` continuations of START for every request: scores and tokens [batch, beams, steps], and the layers'
    states with the beams' slots."""
    sizes, batch = model["sizes"], adapter.shape[0]
    heads, dim, dstate = sizes[1:4]
    slots = torch.arange(batch * beams, device="cuda", dtype=torch.int32).view(batch, beams)
    states = [torch.zeros((batch * beams, heads, dim, dstate), device="cuda") for _ in model["layers"]]
    scores = torch.full((batch, beams), -torch.inf, device="cuda")
    scores[:, 0] = 0  # all beams are the same until the first choice
    finished = torch.zeros((batch, beams), dtype=torch.bool, device="cuda")
    tokens = torch.full((batch, beams), START, device="cuda")
    said = torch.empty((batch, beams, 0), dtype=torch.int64, device="cuda")
    for _ in range(steps):
        logits = step(model, adapters, states, slots, tokens, adapter)
        scores, parents, tokens = ssu.beam_select(logits, scores, beams, finished=finished, end_token=END)
        slots = ssu.reorder_states(states, slots, parents)
        parents, tokens = parents.long().clamp(min=0), tokens.long().clamp(min=0)
        finished = finished.gather(1, parents) | (tokens == END)
        said = torch.cat((said.gather(1, parents[..., None].expand(said.shape)), tokens[..., None]), -1)
    return scores, said, states, slots


# ---------------------------------------------------------------- the same in plain torch


def plain_scores(model, adapters, adapter, said):
    """Scores of given sequences [batch, beams, steps], each with a state of its own."""
    sizes = model["sizes"]
    heads, dim, dstate, groups = sizes[1:5]
    batch, beams, steps = said.shape
    rows = batch * beams
    ids = adapter[:, None].expand(batch, beams).reshape(rows)
    some = (ids >= 0)[:, None]

    def lora(x, pair):
        a, b = (t.float()[ids.clamp(min=0)] for t in pair)
        h = (a @ x[..., None]) * adapters["scale"][ids.clamp(min=0), None, None]
        return torch.where(some, (b @ h)[..., 0], 0.0)
    states = [torch.zeros((rows, heads, dim, dstate), device="cuda") for _ in model["layers"]]
    token = torch.full((rows,), START, device="cuda")
    score = torch.zeros(rows, device="cuda", dtype=torch.float64)
    over = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for t in range(steps):
        x = model["embedding"][token]
        residual = torch.zeros(x.shape, dtype=torch.float32, device="cuda")
        for i, (layer, low) in enumerate(zip(model["layers"], adapters["layers"])):
            residual = residual + x.float()
            h = plain_norm(residual, layer["norm"])
            v = (h @ decode(*layer["in"]).t()).bfloat16().float() + lora(h, low["in"])
            z, xs, B, C, dt = (u.float() for u in split(v.bfloat16(), sizes, rows, 1))
            xs, dt = xs[:, 0], torch.nn.functional.softplus(dt[:, 0] + layer["dt_bias"])
            Bh, Ch = (u[:, 0].repeat_interleave(heads // groups, 1) for u in (B, C))
            s = states[i] * torch.exp(dt * layer["A"])[..., None, None] + (dt[..., None] * xs)[..., None] * Bh[:, :, None]
            states[i] = s
            y = ((s * Ch[:, :, None]).sum(-1) + layer["D"][:, None] * xs).bfloat16().float().reshape(rows, heads * dim)
            g = plain_norm(y * torch.nn.functional.silu(z), layer["gated_norm"], groups)
            x = ((g @ decode(*layer["out"]).t()).bfloat16().float() + lora(g, low["out"])).bfloat16()
        logits = plain_norm(residual + x.float(), model["norm"]) @ decode(*model["head"]).t()
        token = said[:, :, t].reshape(rows)
        gained = torch.log_softmax(logits.double(), -1).gather(1, token[:, None])[:, 0]
        score = score + torch.where(over, 0.0, gained)
        over = over | (token == END)
    return score.view(batch, beams)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--beams", type=int, default=5)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--layers", type=int, default=3)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--vocab", type=int, default=1021)
    ap.add_argument("--rank", type=int, default=8)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    model = make_model(a.layers, a.width, a.heads, 64, 128, 2, a.vocab)
    adapters = make_adapters(model, a.requests, a.rank)
    adapter = torch.arange(a.requests, device="cuda", dtype=torch.int32) - 1  # the first request has none
    scores, said = search(model, adapters, adapter, a.beams, a.steps)[:2]
    for b in range(a.requests):
        print("request %d: score %.3f, tokens %s" % (b, float(scores[b, 0]), said[b, 0].tolist()))
    if not a.check:
        return None
    off = float((plain_scores(model, adapters, adapter, said) - scores).abs().max())
    print("largest difference of a score to plain torch: %.4f over %d steps" % (off, a.steps))
    return off


if __name__ == "__main__":
    main()
