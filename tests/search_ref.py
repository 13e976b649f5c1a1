"""Plain forms of beam_select, reorder_states and add_lora on the CPU, in float64 and
whole numbers, written from their definitions in include/ssu.h."""
import math

import torch

import layer_ref as R


def scores_of(logits, scores, finished=None, end_token=0, mask=None):
    """For every request the list of all its continuations as (score, beam, token, logit), in
    float64; None where something makes the request's answers NaN."""
    batch, beams = scores.shape
    vocab = logits.shape[-1]
    x = logits.reshape(batch, beams, vocab).double()
    out = []
    for b in range(batch):
        found, bad = [], False
        for i in range(beams):
            s = float(scores[b, i])
            if not s < math.inf:
                bad = True
                continue
            if s == -math.inf:
                continue
            if finished is not None and bool(finished[b, i]):
                found.append((s, i, end_token, math.inf))
                continue
            listed = torch.ones(vocab, dtype=torch.bool)
            if mask is not None:
                at = torch.arange(vocab)
                words = mask[0] if mask.shape[0] == 1 else mask[b * beams + i]
                listed = ((words.long()[at // 32] >> (at % 32)) & 1) == 1
            row = x[b, i]
            if bool((listed & ~(row < math.inf)).any()):
                bad = True
                continue
            ids = torch.nonzero(listed & (row > -math.inf))[:, 0]
            if len(ids) == 0:
                continue
            l = row[ids]
            peak = l.max()
            total = torch.log(torch.exp(l - peak).sum())
            found += [(s + float((v - peak) - total), i, int(t), float(v)) for v, t in zip(l, ids)]
        out.append(None if bad else found)
    return out


def beam_select(logits, scores, keep, finished=None, end_token=0, mask=None):
    """(scores in float64, parents, tokens), every one [batch, keep]."""
    s, p, t = [], [], []
    for found in scores_of(logits, scores, finished, end_token, mask):
        if found is None:
            s.append([math.nan] * keep)
            p.append([-1] * keep)
            t.append([-1] * keep)
            continue
        best = sorted(found, key=lambda c: (-c[0], c[1], -c[3], c[2]))[:keep]
        none = keep - len(best)
        s.append([c[0] for c in best] + [-math.inf] * none)
        p.append([c[1] for c in best] + [-1] * none)
        t.append([c[2] for c in best] + [-1] * none)
    return torch.tensor(s, dtype=torch.float64), torch.tensor(p, dtype=torch.int32), torch.tensor(t, dtype=torch.int32)


def reorder(pools, slots, parents):
    """(pools, new slots) of lists and numbers; `pools`: tensors [slots, ...]."""
    before = [p.clone() for p in pools]
    after = [p.clone() for p in pools]
    new = []
    beams = slots.shape[1]
    for mine, par in zip(slots.tolist(), parents.tolist()):
        mine = [m if 0 <= m < 2 ** 31 - 1 else -1 for m in mine]
        par = [q if 0 <= q < beams else -1 for q in par]
        free = [s for i, s in enumerate(mine) if i not in par]
        taken, row = set(), []
        for q in par:
            if q >= 0 and q not in taken:
                row.append(mine[q])
            else:
                to = free.pop(0)
                row.append(to)
                if q >= 0:
                    for a, old in zip(after, before):
                        if 0 <= to < len(a) and 0 <= mine[q] < len(a):
                            a[to] = old[mine[q]]
            if q >= 0:
                taken.add(q)
        assert not free and sorted(row) == sorted(mine)
        new.append(row)
    return after, torch.tensor(new)


def lora(y, x, a, b, adapter, scale=None):
    """(result, allowed error) in float64; x: floats. The error, from its parts:
    - h = x a^T is summed in float32, k/8 + 48 roundings or truncations deep at most (2^-23 each), of sums not above
      sum |x a|;
    - two summands of a 16-bit type hold h to the square of its half step; in float16 the second one is a multiple of
      2^-24 of a power of two not above twice the row's largest h;
    - the sum over the rank, twice as long for two summands, and the addition to y in float32;
    - y's rounding."""
    out, tol = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    dt, k = y.dtype, x.shape[1]
    for i in range(a.shape[0]):
        rows = torch.nonzero(adapter.long() == i)[:, 0]
        if len(rows) == 0:
            continue
        xr, w, v = x[rows].double(), a[i].double(), b[i].double()
        f = 1.0 if scale is None else float(scale[i])
        h, mag = xr @ w.t(), xr.abs() @ w.abs().t()
        dh = (k / 8 + 48) * 2.0 ** -23 * mag + 2.0 ** -24 * h.abs()
        if dt != torch.float32:
            dh = dh + R.ROUND[dt] ** 2 * 2 * h.abs()
        if dt == torch.float16:
            dh = dh + 2.0 ** -24 * h.abs().amax(-1, keepdim=True)
        size = h.abs() @ v.abs().t() * abs(f)
        out[rows] += f * (h @ v.t())
        tol[rows] = dh @ v.abs().t() * abs(f) + (2 * a.shape[1] + 16) * 2.0 ** -23 * size + 2.0 ** -23 * (y[rows].double().abs() + size)
        tol[rows] += R.ROUND[dt] * out[rows].abs() + R.TINY[dt]
    return out, tol
