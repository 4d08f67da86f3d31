"""Oracle for the paged cache (float64, numpy, CPU). Test infrastructure.

[P1] "Motor de inferência Quail atinge 1 bilhão de tokens por minuto por GPU", section
"Como funciona", keeps anchor KV between prefills; here it is kept in pages. Definitions,
with query head h reading KV head g = h // (Hq / Hkv) as everywhere in this package:

  decode   w[h, j] = exp(scale q[h] . k[j, g] - lse[h]) over the cached tokens j,
           out[h] = sum_j w[h, j] v[j, g]; no tokens: out = 0, lse = -inf
  scores   score[g, j] = sum over the queries i that see key j and the heads h of g of
           exp(scale q[i, h] . k[j, g] - lse[i, h]); lse = -inf gives 0
  evict    per KV head: the last `recent` tokens and the largest-scored others, `budget` in
           all, ties to the lower position, NaN as -inf
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_encode


def slots(table_row, positions, page_size):
    """Rows of the flattened pool for positions of one sequence."""
    p = np.asarray(positions, np.int64)
    return np.asarray(table_row, np.int64)[p // page_size] * page_size + p % page_size


def append(pages, new, offsets, start, table, scale=None):
    """pages [P, page, Hkv, d] (values, or e4m3 codes with `scale` [B, Hkv]) with the rows
    new [T, Hkv, d] of each sequence at start[b] ..; returns a copy."""
    out = pages.copy()
    flat = out.reshape(-1, *pages.shape[2:])
    for b in range(len(start)):
        rows = new[offsets[b]:offsets[b + 1]]
        at = slots(table[b], start[b] + np.arange(len(rows)), pages.shape[1])
        if scale is None:
            flat[at] = rows
        else:
            with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
                quotient = rows.astype(np.float32) / scale[b].astype(np.float32)[None, :, None]
            flat[at] = e4m3_encode(quotient)
    return out


def decode(q, k, v, scale):
    """q [Hq, d], k and v [n, Hkv, d] of one sequence -> out [Hq, d], lse [Hq], w [Hkv, n]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    hq, hkv, n = q.shape[0], k.shape[1], k.shape[0]
    group = hq // hkv
    out, lse, w = np.zeros(q.shape), np.full(hq, -np.inf), np.zeros((hkv, n))
    for h in range(hq if n else 0):
        z = scale * (k[:, h // group] @ q[h])
        m = z.max()
        lse[h] = m + np.log(np.exp(z - m).sum())
        p = np.exp(z - lse[h])
        out[h] = p @ v[:, h // group]
        w[h // group] += p
    return out, lse, w


def scores(q, k, lse, scale, causal, window=0):
    """q [nq, Hq, d], k [nk, Hkv, d], lse [nq, Hq] of one sequence -> score [Hkv, nk]."""
    q, k, lse = (np.asarray(x, np.float64) for x in (q, k, lse))
    nq, hq, _ = q.shape
    nk, hkv, _ = k.shape
    total = np.zeros((hkv, nk))
    for i in range(nq - min(window, nq) if window else 0, nq):
        seen = min(nk, max(0, i + nk - nq + 1)) if causal else nk
        for h in range(hq):
            if lse[i, h] != -np.inf:
                g = h // (hq // hkv)
                total[g, :seen] += np.exp(scale * (k[:seen, g] @ q[i, h]) - lse[i, h])
    return total


def evict(score, n, budget, recent):
    """Kept positions (increasing) of one sequence and KV head; score [>= n]."""
    new = min(n, budget)
    last = min(recent, new)
    x = np.asarray(score, np.float64)[:n - last]
    x = np.where(np.isnan(x), -np.inf, x)
    best = np.argsort(-x, kind="stable")[:new - last]
    return np.concatenate([np.sort(best), np.arange(n - last, n)]).astype(np.int64)
