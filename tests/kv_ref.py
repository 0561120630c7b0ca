"""Plain float64 forms of the KV-cache calls on host arrays, with error bounds of the float32 sums."""
from __future__ import annotations

import math

import numpy as np
import torch

EPS32 = 2.0 ** -24          # half a float32 step, relative
# The weights in the product with V.  A chunk of a bfloat16 pool takes them rounded to bfloat16: half a step,
# 2^-8.  One token per sequence takes them as two bfloat16 numbers: the first is the weight cut off to 8 bits, so
# the rest is below 2^-7 of it, and the second is the rest rounded, off by at most 2^-8 of it: 2^-15 in all.
# float32 pools take them as they are.
ROUNDED = {(torch.bfloat16, True): 2.0 ** -8, (torch.bfloat16, False): 2.0 ** -15, (torch.float32, True): 0.0,
           (torch.float32, False): 0.0}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def cached(pages, layout, table_row, n):
    """K and V of one sequence: two [n][n_kv][dim] float64 arrays.  pages: [P][H] tensor (any device); table_row
    [2][max_pages]; tokens of pages outside the pool are absent: also returns which tokens are there."""
    tpp, w = layout.tokens_per_page, layout.n_kv_heads * layout.head_dim
    P = pages.shape[0]
    out, there = [], np.ones(n, bool)
    for r in range(2):
        ids = np.asarray(table_row[r][: -(-n // tpp)]).astype(np.int64)
        ok = (ids >= 0) & (ids < P)
        there &= np.repeat(ok, tpp)[:n]
        rows = pages[torch.as_tensor(np.where(ok, ids, 0), device=pages.device)][:, : tpp * w]
        rows = rows.detach().to("cpu", torch.float32).numpy().astype(np.float64)
        out.append(rows.reshape(-1, layout.n_kv_heads, layout.head_dim)[:n])
    return out[0], out[1], there


def attend(pages, layout, q, table, lens, q_start, scale, rounded):
    """Outputs, bounds on their error before the last rounding, weights summed over rows and heads, and
    their bounds.  q [T][heads * dim] tensor; rows outside every sequence come back as NaN.  rounded: how far the
    weights are off, relatively, in the product with V (ROUNDED)."""
    nh, dim, group = layout.n_heads, layout.head_dim, layout.n_heads // layout.n_kv_heads
    q = q.detach().to("cpu", torch.float32).numpy().astype(np.float64)
    T, n_seq, cap = q.shape[0], len(lens), table.shape[-1] * layout.tokens_per_page
    out, tol = np.full((T, nh * dim), np.nan), np.zeros((T, nh * dim))
    sc, sc_tol = np.zeros((n_seq, cap)), np.zeros((n_seq, cap))
    for b, n in enumerate(lens):
        r0, r1 = (b, b + 1) if q_start is None else (q_start[b], q_start[b + 1])
        if r1 == r0:
            continue
        if n == 0:
            out[r0:r1] = 0
            continue
        K, V, there = cached(pages, layout, table[b], n)
        pos = np.arange(n - (r1 - r0), n)
        seen = (np.arange(n)[None] <= pos[:, None]) & there[None]
        for h in range(nh):
            k, v = K[:, h // group], V[:, h // group]
            qh = q[r0:r1, h * dim:(h + 1) * dim]
            x = np.where(seen, qh @ k.T * scale, -np.inf)
            # a logit: dim products and sums, the scale, and the argument of the exponential, each rounded
            dx = (dim + 4) * EPS32 * abs(scale) * (np.abs(qh) @ np.abs(k).T) + 4 * EPS32 * np.abs(np.where(seen, x, 0))
            dx = np.where(seen, dx, 0).max(1)
            m = x.max(1, keepdims=True)
            e = np.where(seen, np.exp(x - np.where(np.isfinite(m), m, 0)), 0)
            total = e.sum(1, keepdims=True)
            p = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
            # a weight: numerator and denominator off by its logit's error and the exponential's (two steps);
            # sums of n terms, rescaled when the maximum grows; one division
            rel = (2 * dx + (n + 64) * EPS32 + 16 * EPS32)[:, None]
            cols = slice(h * dim, (h + 1) * dim)
            out[r0:r1, cols] = np.where(seen.any(1)[:, None], p @ np.where(there[:, None], v, 0), 0)
            tol[r0:r1, cols] = (rel + rounded) * (p @ np.abs(np.where(there[:, None], v, 0)))
            sc[b, :n] += p.sum(0)
            sc_tol[b, :n] += (p * rel).sum(0)
        sc_tol[b, :n] += sc[b, :n] * (nh * (r1 - r0) + 4) * EPS32
    return out, tol, sc, sc_tol


def evict(layout, table, scores, lens, budget, first, last, max_drop):
    """table [L][n][2][P], scores [L][n][P * tpp] float32 arrays -> what lora_kv_evict returns."""
    tpp, (L, n, _, P) = layout.tokens_per_page, table.shape
    t_out, s_out = np.full_like(table, -1), np.zeros_like(scores)
    lens_out, n_drop = np.array(lens, np.int32), np.zeros(n, np.int32)
    dropped = np.full((L, n, 2, max_drop), -1, np.int32)
    for b, ln in enumerate(lens):
        if ln < 0 or ln > P * tpp:
            t_out[:, b], s_out[:, b] = table[:, b], scores[:, b]
            continue
        can = [i for i in range(-(-ln // tpp)) if i * tpp >= first and (i + 1) * tpp <= ln - last]
        count = min(max_drop, len(can), max(0, -(-(ln - budget) // tpp)))
        n_drop[b], lens_out[b] = count, ln - count * tpp
        for l in range(L):
            def key(i):
                s = float(scores[l, b, i * tpp])
                for j in range(1, tpp):
                    s += float(scores[l, b, i * tpp + j])
                return (math.isnan(s), 0.0 if math.isnan(s) else s, i)
            gone = set(sorted(can, key=key)[:count])
            kept = [i for i in range(-(-ln // tpp)) if i not in gone]
            t_out[l, b, :, : len(kept)] = table[l, b][:, kept]
            toks = [t for t in range(ln) if t // tpp not in gone]
            s_out[l, b, : len(toks)] = scores[l, b, toks]
            dropped[l, b, :, :count] = table[l, b][:, sorted(gone)]
    return t_out, s_out, lens_out, dropped, n_drop
