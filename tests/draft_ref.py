"""Plain forms of the calls of a step of drafted tokens, on the host: Python integers, float64 and error bounds."""
from __future__ import annotations

import numpy as np

import kv_ref
from kv_ref import EPS32


def random_trees(rng, sizes, near=6):
    """Parents, one list behind the other: each node hangs on one of the `near` before it."""
    out = []
    for m in sizes:
        out += [0 if i == 0 else int(rng.integers(max(0, i - near), i)) for i in range(m)]
    return out


def mask_rows(parents, sizes):
    """Python integers: bit j of row i, node i sees node j of its tree."""
    rows, first = [], 0
    for m in sizes:
        for i in range(m):
            rows.append((rows[first + parents[first + i]] if i else 0) | 1 << i)
        first += m
    return rows


def mask_words(rows, words):
    return np.array([[r >> 64 * w & (2 ** 64 - 1) for w in range(words)] for r in rows], np.uint64).reshape(-1, words).view(np.int64)


def attend(pages, layout, q, table, lens, q_start, bits, scale, rounded):
    """Outputs and bounds on their error before the last rounding; rows outside every sequence come back as NaN.
    bits: a Python integer per row of q.  The bounds are kv_ref.attend's, term by term."""
    nh, dim, group = layout.n_heads, layout.head_dim, layout.n_heads // layout.n_kv_heads
    q = q.detach().to("cpu").float().numpy().astype(np.float64)
    out, tol = np.full((q.shape[0], nh * dim), np.nan), np.zeros((q.shape[0], nh * dim))
    for b, n in enumerate(lens):
        r0, r1 = q_start[b], q_start[b + 1]
        if r1 == r0:
            continue
        if n == 0:
            out[r0:r1] = 0
            continue
        K, V, there = kv_ref.cached(pages, layout, table[b], n)
        m = r1 - r0
        seen = np.ones((m, n), bool)
        seen[:, n - m:] = [[bits[r0 + i] >> j & 1 for j in range(m)] for i in range(m)]
        seen &= there[None]
        for h in range(nh):
            k, v = np.where(there[:, None], K[:, h // group], 0), np.where(there[:, None], V[:, h // group], 0)
            qh = q[r0:r1, h * dim:(h + 1) * dim]
            x = np.where(seen, qh @ k.T * scale, -np.inf)
            dx = (dim + 4) * EPS32 * abs(scale) * (np.abs(qh) @ np.abs(k).T) + 4 * EPS32 * np.abs(np.where(seen, x, 0))
            dx = np.where(seen, dx, 0).max(1)
            top = x.max(1, keepdims=True)
            e = np.where(seen, np.exp(x - np.where(np.isfinite(top), top, 0)), 0)
            total = e.sum(1, keepdims=True)
            p = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
            rel = (2 * dx + (n + 64) * EPS32 + 16 * EPS32)[:, None]
            cols = slice(h * dim, (h + 1) * dim)
            out[r0:r1, cols] = np.where(seen.any(1)[:, None], p @ v, 0)
            tol[r0:r1, cols] = (rel + rounded) * (p @ np.abs(v))
    return out, tol


def plan(layers, tpp, counts, lens, held, table, stock, state, T, max_len, parents=None, max_nodes=0, num_pages=1 << 31):
    """What lora_kv_plan writes.  table [L][n][2][P], stock [G][L][2]: copies come back, changed."""
    table, stock = table.copy(), stock.copy()
    n, P, cap = len(counts), table.shape[-1], len(stock)
    head, free = state[:2]
    words = (max_nodes + 63) // 64
    ok_ring = 0 <= head < cap and 0 <= free <= cap
    start_free, room = (free, cap - free) if ok_ring else (0, 0)
    first_free, first_back = (head, (head + free) % cap) if ok_ring else (0, 0)
    out = dict(step_lens=[], q_start=[0], slots=np.full((layers, 2, T), -1, np.int64), positions=np.zeros(T, np.int64),
               mask=np.zeros((T, words), np.uint64), lens=[], held=[])
    taken = asked = back = gave = refused = rows = 0
    err = not ok_ring
    moves = []
    for b in range(n):
        c, ln, h = counts[b], lens[b], held[b]
        if c < 0 or c > (max_nodes if parents is not None else T):
            c, err = 0, True
        valid = 0 <= ln <= max_len and 0 <= h <= P and -(-ln // tpp) <= h
        fits = valid and rows + c <= T and ln + c <= max_len
        err |= not fits
        want = -(-(ln + c) // tpp) if fits else -(-ln // tpp)
        take, give = (max(0, want - h), max(0, h - want)) if valid else (0, 0)
        asked += take
        ok = fits and (take == 0 or asked <= start_free)
        gave += give
        goes = gave <= room
        err |= bool(give) and not goes
        if ok and take:
            for e in range(take):
                moves.append((table, (slice(None), b, slice(None), h + e), stock[(first_free + taken + e) % cap].copy()))
            taken += take
        if give and goes:
            for e in range(h - give, h):
                moves.append((stock, (first_back + back + e - (h - give)) % cap, table[:, b, :, e].copy()))
            back += give
        for target, at, what in moves:
            target[at] = what
        moves = []
        refused += c > 0 and not ok
        out["step_lens"].append(ln + c if ok and c else 0)
        out["lens"].append(ln + c if ok else ln)
        out["held"].append(h + (take if ok else 0) - (give if goes else 0))
        for i in range(c if ok else 0):
            pos, t = ln + i, rows + i
            page = table[:, b, :, pos // tpp].astype(np.int64)
            out["slots"][:, :, t] = np.where((page >= 0) & (page < num_pages), page * tpp + pos % tpp, -1)
            err |= bool(((page < 0) | (page >= num_pages)).any())
            depth, bits, j = i, 0, i
            if parents is not None:
                depth, bits = 0, 1 << i
                while j > 0:
                    up = parents[rows + j]
                    if not 0 <= up < j:
                        err = True
                        break
                    j, depth = up, depth + 1
                    bits |= 1 << j
                out["mask"][t] = [bits >> 64 * w & (2 ** 64 - 1) for w in range(words)]
            out["positions"][t] = ln + depth
        rows += c
        out["q_start"].append(min(rows, T))
    out["state"] = [(head + taken) % cap if ok_ring else head, free - taken + back if ok_ring else free, refused, 0]
    out["table"], out["stock"], out["err"] = table, stock, bool(err)
    return out


def accept(parents, tokens, targets, m, first):
    """The path of one tree whose rows are first .. first + m - 1."""
    path = [0] if m else []
    while m:
        to = [c for c in range(path[-1] + 1, m) if parents[first + c] == path[-1] and tokens[first + c] == targets[first + path[-1]]]
        if not to:
            break
        path.append(to[0])
    return path


def rope(x, table, positions, heads, dim, pairs):
    """x [T][heads * dim] and table [positions][rot / 2][2] float64: rows turned, and bounds on the float32 error: two
    products and a sum, each off by half a step of what they are at most."""
    rot, x = 2 * table.shape[1], x.reshape(-1, heads, dim).copy()
    one = np.arange(0, rot, 2) if pairs else np.arange(rot // 2)
    two = one + (1 if pairs else rot // 2)
    c, s = table[positions][:, None, :, 0], table[positions][:, None, :, 1]
    a, b = x[..., one].copy(), x[..., two].copy()
    tol = np.zeros_like(x)
    x[..., one], x[..., two] = a * c - b * s, a * s + b * c
    tol[..., one] = 3 * EPS32 * (np.abs(a * c) + np.abs(b * s))
    tol[..., two] = 3 * EPS32 * (np.abs(a * s) + np.abs(b * c))
    return x.reshape(len(x), -1), tol.reshape(len(x), -1)
