"""The paged key-value operators, as they are measured: writing new tokens' keys and values into the
pool's pages, attention of one new token per sequence, attention of a chunk of new tokens, and eviction
by accumulated attention weight.  Each has a plain form (elementary torch operations in 32 bits) and the
call of the library; `exact` computes the same outputs in 64 bits.

A page is one vector of `hidden` elements and holds `tpp` tokens of one layer's keys (or values).  A
sequence's table row lists its key pages and its value pages, in token order.
"""
import math
import random

import torch

own = False

# query heads, key/value heads, head dim, hidden, tokens a page holds.  4096 = 32 x 128 and 5120 = 40 x 128
# are the widths of the projection's decode, prefill and 13B-shaped workloads; the others are generic.
GEOMETRY = {
    "h4096": (32, 32, 128, 4096, 1),          # one token's keys fill a page
    "h4096_kv8": (32, 8, 128, 4096, 4),       # shared key heads: four tokens a page
    "h5120": (40, 40, 128, 5120, 1),
    "h5120_kv8": (40, 8, 128, 5120, 5),       # a page count that is no power of two
    "h4096_d256": (16, 4, 256, 4096, 4),
    "h1024_d64": (16, 16, 64, 1024, 1),
    "h1024_d64_kv4": (16, 4, 64, 1024, 4),
    "h1024_mqa": (8, 1, 128, 1024, 7),        # one key head; the page's last eighth stays unused
    "h256_d64": (4, 2, 64, 256, 2),
}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of the 64-token batch: the smallest call, all latency
        dict(name="write_step_64", op="write", geo="h4096", dtype="bf16", n_seq=64, new=1, past=300, ragged=True),
        # the prompts of the prefill workload: 8 x 512 tokens
        dict(name="write_prompt_8x512", op="write", geo="h4096", dtype="bf16", n_seq=8, new=512, past=0, ragged=False),
        # prompts of odd lengths behind a cached prefix, packed pages, float32
        dict(name="write_ragged_f32", op="write", geo="h1024_d64_kv4", dtype="f32", n_seq=13, new=301, past=77, ragged=True),
        # a single user's decode step on a short cache: latency
        dict(name="attend_one", op="attend", geo="h4096", dtype="bf16", n_seq=1, length=203, ragged=False, scores=False),
        # the 64-token decode batch on caches of mixed length, weights collected for eviction
        dict(name="attend_64", op="attend", geo="h4096", dtype="bf16", n_seq=64, length=1031, ragged=True, scores=True),
        # long caches with shared key heads: split over the length
        dict(name="attend_long_kv8", op="attend", geo="h4096_kv8", dtype="bf16", n_seq=8, length=32768, ragged=True, scores=True),
        # float32 pool, small heads
        dict(name="attend_f32", op="attend", geo="h1024_d64", dtype="f32", n_seq=16, length=777, ragged=True, scores=False),
        # the prefill workload's prompts, weights collected for eviction
        dict(name="chunk_prompt_8x512", op="chunk", geo="h4096", dtype="bf16", n_seq=8, new=512, past=0, ragged=False, scores=True),
        # the last 2048 tokens of a 16384-token prompt, taken chunk by chunk, shared key heads
        dict(name="chunk_extend_16k", op="chunk", geo="h4096_kv8", dtype="bf16", n_seq=1, new=2048, past=14336, ragged=False, scores=False),
        # float32, odd lengths, some tokens cached before
        dict(name="chunk_ragged_f32", op="chunk", geo="h1024_d64", dtype="f32", n_seq=5, new=201, past=130, ragged=True, scores=True),
        # all 32 layers of 16 requests cut back to half of 4096 tokens
        dict(name="evict_32_layers", op="evict", geo="h4096", dtype="bf16", layers=32, n_seq=16, length=4096, ragged=True, budget=2048),
        # one layer of a few packed caches: latency
        dict(name="evict_packed", op="evict", geo="h5120_kv8", dtype="bf16", layers=1, n_seq=4, length=2003, ragged=True, budget=1500),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "chunk", "chunk", "evict"])
    geo = rng.choice(sorted(GEOMETRY))
    heads, kv, dim, hidden, tpp = GEOMETRY[geo]
    case = dict(op=op, geo=geo, dtype=rng.choice(["bf16", "bf16", "f32"]), ragged=rng.random() < 0.7)
    size = (2 if case["dtype"] == "bf16" else 4) * kv * dim
    if op == "write":
        n = _log(rng, 1, 256)
        case.update(n_seq=n, new=_log(rng, 1, max(1, min(1024, 2 ** 25 // (n * size)))), past=_log(rng, 1, 600) - 1)
    elif op == "attend":
        n = _log(rng, 1, 256)
        case.update(n_seq=n, length=_log(rng, 1, max(2, min(32768, 2 ** 29 // (2 * n * size)))), scores=rng.random() < 0.5)
    elif op == "chunk":
        most = 2 ** 36 if case["dtype"] == "bf16" else 2 ** 31            # multiply-adds of one product, before the mask
        n = _log(rng, 1, 16)
        new = _log(rng, 1, min(2048, int(math.sqrt(most / (n * heads * dim)))))
        past = _log(rng, 1, max(1, min(14336, most // (n * heads * dim * new)))) - 1
        case.update(n_seq=n, new=new, past=past, scores=rng.random() < 0.5)
    else:
        layers, n = _log(rng, 1, 40), _log(rng, 1, 64)
        length = _log(rng, 1, min(32768, 2 ** 21 // (layers * n)))
        case.update(layers=layers, n_seq=n, length=length, budget=rng.randint(1, length + 1))
    return case


def _between(case, key, most, least):
    """One number per sequence: all `most`, or spread over [least, most] with `most` among them."""
    n = case["n_seq"]
    if not case["ragged"]:
        return [most] * n
    r = random.Random("%s %d %d %d" % (key, n, most, least))
    got = [r.randint(least, most) for _ in range(n)]
    got[r.randrange(n)] = most
    return got


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    if case["op"] in ("write", "chunk"):
        new = _between(case, "new", case["new"], (case["new"] + 3) // 4)
        past = _between(case, "past", case["past"], case["past"] // 4)
        return new, [a + b for a, b in zip(new, past)]
    total = _between(case, "len", case["length"], (case["length"] + 3) // 4)
    return [1] * case["n_seq"], total


def _ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def prepare(case, seed):
    heads, kv, dim, hidden, tpp = GEOMETRY[case["geo"]]
    dt, n_seq, op = DTYPE[case["dtype"]], case["n_seq"], case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, total = _lengths(case)
    layers = case.get("layers", 1)
    width = (max(total) + tpp - 1) // tpp                                  # table entries of a sequence
    s = dict(case=case, heads=heads, kv=kv, dim=dim, hidden=hidden, tpp=tpp, width=width, scale=dim ** -0.5,
             longest=max(total), lens=_ints(total), T=sum(new), new=max(new))
    # tables: every sequence has its own pages, placed at random, -1 behind its last
    held = torch.arange(width, device="cuda")[None, :] < ((s["lens"] + tpp - 1) // tpp)[:, None]
    n_pages = int(2 * layers * held.sum())
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((layers, n_seq, 2, width), -1, dtype=torch.int32, device="cuda")
    table[held[None, :, None, :].expand_as(table)] = order
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    s["starts"] = _ints(starts)
    s["table"] = table if op == "evict" else table[0]
    if op == "evict":
        # accumulated weights: most tokens little, a few much, and some never looked at (ties at zero)
        w = torch.rand((layers, n_seq, width * tpp), generator=g, device="cuda")
        s["scores"] = torch.where(w < 0.1, torch.zeros_like(w), w ** 4 * 30)
        s.update(budget=case["budget"], first=4, last=min(64, case["length"] // 4), drop=width)
        pages = torch.empty((16, hidden), dtype=dt, device="cuda")
    else:
        pages = torch.empty((n_pages, hidden), dtype=dt, device="cuda").normal_(generator=g)
    if op == "write":
        rows = torch.empty((s["T"], 2, kv * dim), dtype=dt, device="cuda").normal_(generator=g)
        s["k"], s["v"] = rows[:, 0], rows[:, 1]                            # one projection's output, two column ranges
    if op in ("attend", "chunk"):
        # twice the unit variance: logits of a few units, so that some tokens carry most of the weight
        s["q"] = torch.empty((s["T"], heads * dim), dtype=dt, device="cuda").normal_(generator=g) * 2
        s["scores"] = torch.rand((n_seq, width * tpp), generator=g, device="cuda") if case["scores"] else None
        s["summed"] = torch.zeros_like(s["scores"]) if case["scores"] else None   # zero behind a sequence's last token
    if own:
        import rank_gemm_unified_amd as rg
        s["pool"] = rg.Pool(len(pages), hidden, rg.LORA_BF16 if dt is torch.bfloat16 else rg.LORA_F32, max_rank=1)
        s["pool"].pages.copy_(pages)
        pages = s["pool"].pages
        s["layout"] = rg.lora_kv_layout_t(heads, kv, dim, tpp)
    s["pages"] = pages
    return s


def run(s):
    return {"write": _write, "attend": _attend, "chunk": _chunk, "evict": _evict}[s["case"]["op"]](s)


# ---- the calls of the library, each with its plain form --------------------------------------------------

def _tokens(s):
    """Sequence and position of each new token, from the starts and the lengths."""
    starts, lens = s["starts"].long(), s["lens"].long()
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    return b, t - starts[b] + lens[b] - (starts[1:] - starts[:-1])[b]


def _write(s):
    if own:
        s["pool"].kv_write(s["layout"], s["k"], s["v"], s["table"], s["lens"], s["starts"])
        return s["pages"]
    tpp, w = s["tpp"], s["kv"] * s["dim"]
    b, pos = _tokens(s)
    held = s["pages"][:, : tpp * w].unflatten(1, (tpp, w))
    held[s["table"][b, 0, pos // tpp].long(), pos % tpp] = s["k"]
    held[s["table"][b, 1, pos // tpp].long(), pos % tpp] = s["v"]
    return s["pages"]


def _cached(s):
    """Keys and values in 32 bits, [n_seq][kv heads][tokens][dim]; tokens behind a sequence's last are zero."""
    tpp, w = s["tpp"], s["kv"] * s["dim"]
    kv = s["pages"][s["table"].clamp(min=0).long()][..., : tpp * w].float()
    kv = kv.reshape(len(s["lens"]), 2, -1, s["kv"], s["dim"])[:, :, : s["longest"]]
    there = torch.arange(kv.shape[2], device="cuda") < s["lens"][:, None]
    kv = kv * there[:, None, :, None, None]
    return kv[:, 0].transpose(1, 2).contiguous(), kv[:, 1].transpose(1, 2).contiguous(), there


def _softmax(x, seen):
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0)


def _add_scores(s, weights, there):
    """weights [n_seq][tokens]: the scores of the tokens that a sequence holds, with them; the others stay."""
    old = s["summed"][:, : weights.shape[1]]
    s["summed"][:, : weights.shape[1]] = torch.where(there, s["scores"][:, : weights.shape[1]] + weights, old)
    return s["summed"]


def _attend(s):
    if own:
        o = s["pool"].kv_attend(s["layout"], s["q"], s["table"], s["lens"], scale=s["scale"], max_len=s["longest"],
                                scores=s["summed"], prior=s["scores"])
        return [o] if s["scores"] is None else [o, s["summed"]]
    k, v, there = _cached(s)
    n = len(s["lens"])
    q = s["q"].float().reshape(n, s["kv"], -1, s["dim"])
    p = _softmax(torch.matmul(q, k.transpose(2, 3)) * s["scale"], there[:, None, None, :])
    o = torch.matmul(p, v).reshape(n, -1).to(s["q"].dtype)
    return [o] if s["scores"] is None else [o, _add_scores(s, p.sum((1, 2)), there)]


def _chunk(s):
    if own:
        o = s["pool"].kv_attend_chunk(s["layout"], s["q"], s["table"], s["lens"], s["starts"], scale=s["scale"],
                                      max_len=s["longest"], scores=s["summed"], prior=s["scores"])
        return [o] if s["scores"] is None else [o, s["summed"]]
    k, v, there = _cached(s)
    n, group = len(s["lens"]), s["heads"] // s["kv"]
    b, pos = _tokens(s)
    row = torch.arange(s["T"], device="cuda") - s["starts"].long()[b]
    q = torch.zeros((n, s["new"], s["kv"], group, s["dim"]), device="cuda")
    q[b, row] = s["q"].float().reshape(-1, s["kv"], group, s["dim"])
    at = torch.full((n, s["new"]), -1, device="cuda")
    at[b, row] = pos
    q = q.permute(0, 2, 3, 1, 4).reshape(n, s["kv"], -1, s["dim"])          # rows: (head of the group, new token)
    x = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).unflatten(2, (group, -1))
    seen = torch.arange(k.shape[2], device="cuda") <= at[:, :, None]
    p = _softmax(x, seen[:, None, None])
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (group, -1)).permute(0, 3, 1, 2, 4)
    o = o[b, row].reshape(s["T"], -1).to(s["q"].dtype)
    return [o] if s["scores"] is None else [o, _add_scores(s, p.sum((1, 2, 3)), there)]


def _evict(s):
    if own:
        return s["pool"].kv_evict(s["layout"], s["table"], s["scores"], s["lens"], s["budget"], keep_first=s["first"],
                                  keep_last=s["last"], max_drop=s["drop"])
    tpp, width, lens = s["tpp"], s["width"], s["lens"].long()
    token = s["scores"].unflatten(2, (width, tpp))                         # [layers][n_seq][pages][tokens]
    total = token.double().sum(-1)                             # in 64 bits: two pages' sums may lie close
    page = torch.arange(width, device="cuda")
    free = (page * tpp >= s["first"]) & ((page + 1) * tpp <= (lens - s["last"])[:, None])
    drop = torch.minimum((lens - s["budget"] + tpp - 1).clamp(min=0) // tpp, free.sum(1)).clamp(max=s["drop"])
    rank = torch.where(free, total, math.inf).sort(dim=2, stable=True).indices.argsort(dim=2)
    gone = rank < drop[:, None]
    held = page < ((lens + tpp - 1) // tpp)[:, None]
    order = torch.where(gone, 1, torch.where(held, 0, 2)).sort(dim=2, stable=True).indices
    left = lens - drop * tpp
    table = s["table"].gather(3, order[:, :, None].expand_as(s["table"]))
    table = torch.where((page < ((left + tpp - 1) // tpp)[:, None])[:, None], table, -1)
    scores = token.gather(2, order[..., None].expand_as(token)).flatten(2)
    scores = torch.where(torch.arange(width * tpp, device="cuda") < left[:, None], scores, 0.0)
    first = torch.where(gone, 0, 1).sort(dim=2, stable=True).indices[:, :, : s["drop"]]
    dropped = s["table"].gather(3, first[:, :, None].expand(-1, -1, 2, -1))
    dropped = torch.where((page[: s["drop"]] < drop[:, None])[:, None], dropped, -1)
    return table, scores, left.int(), dropped, drop.int()


# ---- the operators' definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "attend": _exact_rows, "chunk": _exact_rows, "evict": _exact_evict}[case["op"]](s)


def _exact_write(s):
    """What is copied has no rounding: the pages, filled sequence by sequence."""
    pages, w = s["pages"].double(), s["kv"] * s["dim"]
    starts, lens, table = s["starts"].tolist(), s["lens"].tolist(), s["table"].cpu().numpy()
    where = [[], []]
    offset = []
    for b, n in enumerate(lens):
        for t in range(n - (starts[b + 1] - starts[b]), n):
            where[0].append(int(table[b, 0, t // s["tpp"]]))
            where[1].append(int(table[b, 1, t // s["tpp"]]))
            offset.append(t % s["tpp"] * w)
    offset = torch.tensor(offset, device="cuda")
    for which, rows in enumerate((s["k"], s["v"])):
        at = torch.tensor(where[which], device="cuda") * s["hidden"] + offset
        for first in range(0, len(at), 1024):                              # flat addresses, a part at a time
            flat = at[first: first + 1024, None] + torch.arange(w, device="cuda")
            pages.view(-1)[flat.reshape(-1)] = rows[first: first + 1024].double().reshape(-1)
    return pages


def _exact_rows(s):
    """Attention of each sequence's new tokens, head by head of the shared ones, over its own pages alone."""
    kv, dim, tpp, group = s["kv"], s["dim"], s["tpp"], s["heads"] // s["kv"]
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    out = torch.zeros((s["T"], s["heads"], dim), dtype=torch.float64, device="cuda")
    scores = None if s["scores"] is None else torch.zeros(s["scores"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        count = (n + tpp - 1) // tpp
        rows = s["pages"][s["table"][b, :, :count].reshape(-1).long(), : tpp * kv * dim]
        rows = rows.reshape(2, count * tpp, kv, dim)[:, :n].double()
        position = torch.arange(n - (last - first), n, device="cuda")
        future = torch.arange(n, device="cuda")[None, :] > position[:, None]
        if scores is not None:
            scores[b, :n] = s["scores"][b, :n].double()
        for j in range(kv):
            for h in range(j * group, (j + 1) * group):
                q = s["q"][first:last, h * dim: (h + 1) * dim].double()
                x = (q @ rows[0, :, j].T) * s["scale"]
                p = torch.softmax(x.masked_fill(future, -math.inf), dim=1)
                out[first:last, h] = p @ rows[1, :, j]
                if scores is not None:
                    scores[b, :n] += p.sum(0)
    out = out.reshape(s["T"], -1)
    return [out] if scores is None else [out, scores]


def _exact_evict(s):
    """Row by row on the host; only the scores are computed numbers, and they are moved, not changed."""
    tpp, width = s["tpp"], s["width"]
    scores = s["scores"].double().cpu()
    out = torch.zeros_like(scores)
    for layer in range(scores.shape[0]):
        for b, n in enumerate(s["lens"].tolist()):
            row = scores[layer, b].tolist()
            low = -(-s["first"] // tpp)
            sums = []
            for i in range(low, max(low, (n - s["last"]) // tpp)):
                total = 0.0
                for v in row[i * tpp: (i + 1) * tpp]:
                    total += v
                sums.append((total, i))
            count = min(s["drop"], len(sums), max(0, -(-(n - s["budget"]) // tpp)))
            gone = {i for _, i in sorted(sums)[:count]}
            kept = [row[t] for t in range(n) if t // tpp not in gone]
            out[layer, b, : len(kept)] = torch.tensor(kept, dtype=torch.float64)
    return None, out.cuda(), None, None, None


def work(case):
    """Each input read once, each output written once; products and sums of attention alone."""
    heads, kv, dim, hidden, tpp = GEOMETRY[case["geo"]]
    size = 2 if case["dtype"] == "bf16" else 4
    new, total = _lengths(case)
    T, pages = sum(new), sum((n + tpp - 1) // tpp for n in total)
    if case["op"] == "write":
        touched = sum((n - 1) // tpp - (n - m) // tpp + 1 for m, n in zip(new, total))
        return {"bytes": 4 * T * kv * dim * size + 8 * touched, "flops": 0}
    if case["op"] == "evict":
        return {"bytes": case["layers"] * (2 * 8 * pages + 2 * 4 * sum(total)), "flops": 0}
    rows = sum(sum(range(n - m + 1, n + 1)) for m, n in zip(new, total))     # (row, token) pairs that the mask lets through
    moved = 2 * sum(total) * kv * dim * size + 8 * pages + 2 * T * heads * dim * size
    if case["scores"]:
        moved += 2 * 4 * sum(total)
    return {"bytes": moved, "flops": 4 * rows * heads * dim}
