"""The operators of a step of drafted tokens over the paged cache, as they are measured: planning the step on the
GPU (pages, slots, positions and masks from lengths), writing its rows with rotary embedding, attention of a tree
of drafted tokens, and keeping the accepted path.  Each has a plain form (elementary torch operations in 32 bits)
and the call of the library; `exact` computes the same numbers in 64 bits.

A page is one vector of `hidden` elements and holds `tpp` tokens of one layer's keys (or values).  A sequence's
table row lists its key pages and its value pages, in token order.  A drafted tree's nodes are a sequence's last
tokens; node 0 is the root, and a node comes behind its parent.
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
        # one decode step of the 64-token batch in 32 layers, some sequences shortened by the step before: latency
        dict(name="plan_step_64", op="plan", geo="h4096", layers=32, n_seq=64, length=1031, new=1, tree=False, ragged=True, short=False),
        # the same batch with trees of 16 drafted tokens, packed pages
        dict(name="plan_tree_64", op="plan", geo="h4096_kv8", layers=32, n_seq=64, length=1031, new=16, tree=True, ragged=True, short=False),
        # the prefill workload's prompts, 8 x 512 tokens in 32 layers, more than the free pages hold
        dict(name="plan_prompt_8x512", op="plan", geo="h4096", layers=32, n_seq=8, length=40, new=512, tree=False, ragged=False, short=True),
        # one layer's rows of a decode step, 64 tokens: latency
        dict(name="rope_step_64", op="rope", geo="h4096", dtype="bf16", T=64, pad=0, rot=128, pairs=False, far=1031),
        # the prefill workload's 8 x 512 tokens
        dict(name="rope_prompt_8x512", op="rope", geo="h4096", dtype="bf16", T=4096, pad=0, rot=128, pairs=False, far=512),
        # float32, packed pages, half of each head turned, neighbouring elements paired, some rows of padding
        dict(name="rope_half_f32", op="rope", geo="h1024_d64_kv4", dtype="f32", T=2311, pad=97, rot=32, pairs=True, far=9001),
        # a single user's tree of 16 drafted tokens on a short cache: latency
        dict(name="tree_one", op="tree", geo="h4096", dtype="bf16", n_seq=1, length=203, new=16, ragged=False),
        # trees of 16 on the 64-token decode batch's caches of mixed length
        dict(name="tree_64", op="tree", geo="h4096", dtype="bf16", n_seq=64, length=1031, new=16, ragged=True),
        # trees of 32 on long caches with shared key heads
        dict(name="tree_long_kv8", op="tree", geo="h4096_kv8", dtype="bf16", n_seq=8, length=32768, new=32, ragged=True),
        # float32 pool, small heads, trees of odd sizes
        dict(name="tree_f32", op="tree", geo="h1024_d64", dtype="f32", n_seq=16, length=777, new=13, ragged=True),
        # one user's four drafts of five tokens, 40 layers, packed pages: latency
        dict(name="accept_one", op="accept", geo="h5120_kv8", dtype="bf16", layers=40, n_seq=1, past=203, chains=4, depth=5, ragged=False),
        # the 64-token batch, three drafts of five tokens each, 32 layers
        dict(name="accept_64", op="accept", geo="h4096", dtype="bf16", layers=32, n_seq=64, past=20, chains=3, depth=5, ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "tree", "tree", "accept"])
    geo = rng.choice(sorted(GEOMETRY))
    heads, kv, dim, hidden, tpp = GEOMETRY[geo]
    case = dict(op=op, geo=geo)
    if op != "plan":
        case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "plan":
        layers, n, tree = _log(rng, 1, 40), _log(rng, 1, 256), rng.random() < 0.5
        new = _log(rng, 1, max(1, min(64 if tree else 1024, 2 ** 17 // (layers * n))))
        length = _log(rng, 1, max(1, min(8192, 2 ** 20 // (layers * n))))
        case.update(layers=layers, n_seq=n, length=length, new=new, tree=tree, ragged=rng.random() < 0.7, short=rng.random() < 0.3)
    elif op == "rope":
        T = _log(rng, 1, max(2, min(8192, 2 ** 25 // (heads * dim * size))))
        rot = rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= dim])
        case.update(T=T, pad=rng.choice([0, 0, 1, 37]), rot=rot, pairs=rng.random() < 0.5, far=_log(rng, 1, 16384))
    elif op == "tree":
        n = _log(rng, 1, 128)
        new = _log(rng, 1, min(100, 2 ** 14 // (n * heads)) if n * heads <= 2 ** 14 else 1)
        most = min(32768, 2 ** 29 // (2 * n * size * kv * dim), 2 ** (28 if size == 2 else 25) // (n * heads * new))
        case.update(n_seq=n, length=_log(rng, 1, max(2, most)), new=new, ragged=rng.random() < 0.7)
    else:
        layers, n = _log(rng, 1, 40), _log(rng, 1, 64)
        chains = rng.randint(1, 6)
        depth = _log(rng, 1, max(1, min(12, 2 ** 28 // (layers * n * chains * 2 * size * kv * dim * 2))))
        case.update(layers=layers, n_seq=n, past=_log(rng, 1, 300) - 1, chains=chains, depth=depth, ragged=rng.random() < 0.7)
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


def _sum_to(counts):
    starts = [0]
    for m in counts:
        starts.append(starts[-1] + m)
    return starts


def _pages(tokens, tpp):
    return (tokens + tpp - 1) // tpp


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _trees(counts, seed):
    """Parents of each tree's nodes: a node hangs on one of the few before it, the nearest ones more often."""
    r = random.Random(seed)
    return [i - 1 - int(r.random() ** 2 * min(i, 6)) if i else 0 for m in counts for i in range(m)]


def prepare(case, seed):
    heads, kv, dim, hidden, tpp = GEOMETRY[case["geo"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case, heads=heads, kv=kv, dim=dim, hidden=hidden, tpp=tpp, scale=dim ** -0.5, dt=DTYPE.get(case.get("dtype")))
    {"plan": _prepare_plan, "rope": _prepare_rope, "tree": _prepare_tree, "accept": _prepare_accept}[case["op"]](s, case, g, seed)
    if own:
        import rank_gemm_unified_amd as rg
        s["pool"] = rg.Pool(s["n_pages"], hidden, rg.LORA_F32 if s["dt"] is torch.float32 else rg.LORA_BF16, max_rank=1)
        if "pages" in s:
            s["pool"].pages.copy_(s["pages"])
            s["pages"] = s["pool"].pages
        s["layout"] = rg.lora_kv_layout_t(heads, kv, dim, tpp)
        if case["op"] == "rope":
            s["rope"] = rg.Rope(s["turn"], interleaved=case["pairs"])
        elif case["op"] == "plan":
            s["plan"] = rg.KvPlan(*s["out"])
        elif case["op"] == "accept":
            s["kept"] = rg.KvAccepted(*s["out"])
    return s


def run(s):
    return {"plan": _plan, "rope": _rope, "tree": _tree, "accept": _accept}[s["case"]["op"]](s)


def exact(case, seed):
    if case["op"] == "plan":
        return None                                          # whole numbers alone
    s = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "accept": _exact_accept}[case["op"]](s)


def _closure(step):
    """Boolean [n][m][m], each row with at most one entry: what is reached from each node by any number of steps."""
    m = step.shape[-1]
    reach = (step | torch.eye(m, dtype=torch.bool, device="cuda")).float()
    for _ in range(max(1, (m - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    return reach > 0


def _padded(s, rows, fill):
    """A number per row as [n_seq][most rows of one]."""
    b, at = s["of"]
    out = torch.full((s["case"]["n_seq"], s["most"]), fill, dtype=torch.int64, device="cuda")
    out[b, at] = rows.long()
    return out


def _rows_of(s, counts):
    s["of"] = (_ints([b for b, m in enumerate(counts) for _ in range(m)], torch.int64),
               _ints([i for m in counts for i in range(m)], torch.int64))
    s["most"] = max(counts)


# ---- planning a step: tables, slots, positions and masks from lengths -------------------------------------------

def _plan_sizes(case):
    """Per sequence: tokens cached, new ones, pages held (some have more than their tokens need)."""
    tpp = GEOMETRY[case["geo"]][4]
    lens = _between(case, "len", case["length"], case["length"] // 4)
    new = _between(case, "new", case["new"], (case["new"] + 1) // 2 if case["tree"] else case["new"])
    spare = _between(dict(case, ragged=True), "spare", 7, 0)
    return lens, new, [_pages(n + (x if b % 3 == 0 else 0), tpp) for b, (n, x) in enumerate(zip(lens, spare))]


def _prepare_plan(s, case, g, seed):
    tpp, layers, n = s["tpp"], case["layers"], case["n_seq"]
    lens, new, held = _plan_sizes(case)
    want = [_pages(a + b, tpp) for a, b in zip(lens, new)]
    width = max(max(want), max(held))
    need = sum(max(0, w - h) for w, h in zip(want, held))
    free = need - (need + 7) // 8 if case["short"] else need + 5
    groups = sum(held) + free                                # what there is: held by sequences, and free
    s["n_pages"] = 2 * layers * groups
    ids = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32).reshape(groups, layers, 2)
    table = torch.full((layers, n, 2, width), -1, dtype=torch.int32, device="cuda")
    there = torch.arange(width, device="cuda") < _ints(held)[:, None]
    b, e = there.nonzero(as_tuple=True)
    table[:, b, :, e] = ids[: sum(held)]
    s["table"], s["width"], s["T"] = table, width, sum(new) + (3 if case["ragged"] else 0)
    head = seed % groups                                     # the free ones lie anywhere in the ring
    s["stock"] = torch.roll(torch.cat([ids[sum(held):], torch.full_like(ids[: sum(held)], -1)]), head, 0).contiguous()
    s["lens"], s["held"], s["counts"], s["state"] = _ints(lens), _ints(held), _ints(new), _ints([head, free, 0, 0])
    s["parents"] = _ints(_trees(new, seed) + [0] * (s["T"] - sum(new))) if case["tree"] else None
    s["nodes"] = case["new"] if case["tree"] else 0
    s["most"] = max(new)
    T, z = s["T"], dict(dtype=torch.int32, device="cuda")
    s["out"] = (torch.empty(n, **z), torch.empty(n + 1, **z), torch.empty((layers, 2, T), dtype=torch.int64, device="cuda"),
                torch.empty(T, **z), torch.empty((T, _pages(s["nodes"], 64)), dtype=torch.int64, device="cuda") if case["tree"] else None,
                torch.empty(n, **z), torch.empty(n, **z), torch.empty(4, **z))


def _plan(s):
    if own:
        p = s["pool"].kv_plan(s["layout"], s["counts"], s["lens"], s["held"], s["table"], s["stock"], s["state"], s["T"],
                              parents=s["parents"], max_nodes=s["nodes"], out=s["plan"])
        return [p.step_lens, p.q_start, p.slots, p.positions, p.lens, p.held, p.state, s["table"], s["stock"]] + \
            ([] if p.mask is None else [p.mask])
    tpp, T, n, width, cap = s["tpp"], s["T"], len(s["lens"]), s["width"], len(s["stock"])
    lens, held, counts, state = s["lens"].long(), s["held"].long(), s["counts"].long(), s["state"].long()
    want = (lens + counts + tpp - 1) // tpp
    take = (want - held).clamp(min=0)
    upto = take.cumsum(0)
    ok = (take == 0) | (upto <= state[1])
    give = torch.where(ok, (held - want).clamp(min=0), 0)
    # pages that come: entries [held, want) of the sequences that are served
    e = torch.arange(width, device="cuda")
    comes = ok[:, None] & (e >= held[:, None]) & (e < want[:, None])
    which = (state[0] + (upto - take)[:, None] + e - held[:, None]) % cap
    fresh = s["stock"][which].permute(2, 0, 3, 1)
    s["table"].copy_(torch.where(comes[None, :, None, :], fresh, s["table"]))
    # pages that go: entries [want, held), behind the free ones
    goes = ok[:, None] & (e >= want[:, None]) & (e < held[:, None])
    b, at = goes.nonzero(as_tuple=True)
    to = (state[0] + state[1] + (give.cumsum(0) - give)[b] + at - want[b]) % cap
    s["stock"][to] = s["table"][:, b, :, at]
    # rows
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)])
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    real = b < n
    b = b.clamp(max=n - 1)
    real &= ok[b]
    i = t - starts[b]
    pos = lens[b] + i
    at = torch.where(real, pos // tpp, 0)
    slots = torch.where(real[:, None, None], s["table"][:, b, :, at].long() * tpp + (pos % tpp)[:, None, None], -1)
    step = torch.where(ok & (counts > 0), lens + counts, 0)
    mask, where = [], pos
    if s["parents"] is not None:
        m = s["most"]
        par = torch.full((n, m + 1), -1, dtype=torch.int64, device="cuda")
        j = torch.where(real, i, m)                          # rows of no tree: a column of their own
        par[b, j] = torch.where(j > 0, s["parents"].long(), -1)
        seen = _closure(par[:, :m, None] == torch.arange(m, device="cuda"))
        where = lens[b] + seen[b, j.clamp(max=m - 1)].sum(-1) - 1
        words = (s["nodes"] + 63) // 64
        bits = torch.zeros((n, m, words * 64), dtype=torch.int64, device="cuda")
        bits[..., :m] = seen
        bits = (bits.unflatten(2, (words, 64)) << torch.arange(64, device="cuda")).sum(-1)
        mask = [torch.where(real[:, None], bits[b, j.clamp(max=m - 1)], 0)]
    taken = torch.where(ok & (take > 0), upto, 0).max()
    state = torch.stack([(state[0] + taken) % cap, state[1] - taken + give.sum(), (~ok).sum(), state[3]])
    return [step.int(), starts.int(), slots.permute(1, 2, 0), torch.where(real, where, 0).int(), torch.where(ok, lens + counts, lens).int(),
            torch.where(ok, want, held).int(), state.int(), s["table"], s["stock"]] + mask


# ---- rotary embedding, and the rows into their slots -------------------------------------------------------------

def _prepare_rope(s, case, g, seed):
    T, tpp, dt = case["T"] + case["pad"], s["tpp"], s["dt"]
    s["n_pages"] = 2 * _pages(case["T"], tpp) + 3
    s["pages"] = torch.empty((s["n_pages"], s["hidden"]), dtype=dt, device="cuda").normal_(generator=g)
    slots = torch.full((2, T), -1, dtype=torch.int64, device="cuda")
    slots[:, : case["T"]] = torch.randperm(s["n_pages"] * tpp, generator=g, device="cuda")[: 2 * case["T"]].reshape(2, -1)
    s["slots"] = slots
    far = case["far"]
    s["positions"] = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
    angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    s["turn"] = torch.stack([angle.cos(), angle.sin()], -1).float()          # [position][pair][cosine, sine]
    w, k = s["heads"] * s["dim"], s["kv"] * s["dim"]
    rows = torch.empty((T, w + 2 * k), dtype=dt, device="cuda").normal_(generator=g)
    s["q"], s["k"], s["v"] = rows[:, :w], rows[:, w: w + k], rows[:, w + k:]  # one projection's output
    s["q_out"] = torch.zeros((T, w), dtype=dt, device="cuda")


def _turned(s, x):
    rot = s["case"]["rot"]
    x = x.float().unflatten(1, (-1, s["dim"]))
    c, d = s["turn"][s["positions"].long()][:, None].unbind(-1)
    if s["case"]["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * d, a * d + b * c], -1).flatten(2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * c - b * d, a * d + b * c], -1)
    return torch.cat([y, x[..., rot:]], -1).flatten(1).to(s["dt"])


def _rope(s):
    if own:
        s["pool"].kv_write_rope(s["layout"], s["rope"], s["q"], s["k"], s["v"], s["slots"], s["positions"], q_out=s["q_out"])
        return [s["q_out"], s["pages"]]
    tpp, w = s["tpp"], s["kv"] * s["dim"]
    real = (s["slots"] >= 0).all(0)
    s["q_out"].copy_(torch.where(real[:, None], _turned(s, s["q"]), s["q_out"]))
    held = s["pages"][:, : tpp * w].unflatten(1, (tpp, w))
    k, v = s["slots"][0][real], s["slots"][1][real]
    held[k // tpp, k % tpp] = _turned(s, s["k"])[real]
    held[v // tpp, v % tpp] = s["v"][real]
    return [s["q_out"], s["pages"]]


def _exact_rope(s):
    """By complex numbers, a head at a time; the pages filled row by row through flat addresses."""
    rot, dim, w = s["case"]["rot"], s["dim"], s["kv"] * s["dim"]
    T = s["case"]["T"]
    turn = torch.view_as_complex(s["turn"][s["positions"][:T].long()].double().contiguous())
    at = torch.arange(rot // 2, device="cuda")
    one, two = (2 * at, 2 * at + 1) if s["case"]["pairs"] else (at, at + rot // 2)

    def rotate(x, heads):
        x = x[:T].double()
        for h in range(heads):
            z = torch.complex(x[:, h * dim + one], x[:, h * dim + two]) * turn
            x[:, h * dim + one], x[:, h * dim + two] = z.real, z.imag
        return x

    q = s["q_out"].double()
    q[:T] = rotate(s["q"], s["heads"])
    pages = s["pages"].double()
    for slots, rows in ((s["slots"][0], rotate(s["k"], s["kv"])), (s["slots"][1], s["v"][:T].double())):
        first = slots[:T] // s["tpp"] * s["hidden"] + slots[:T] % s["tpp"] * w
        for i in range(0, T, 1024):
            pages.view(-1)[(first[i: i + 1024, None] + torch.arange(w, device="cuda")).reshape(-1)] = rows[i: i + 1024].reshape(-1)
    return [q, pages]


# ---- attention of a tree of new tokens ------------------------------------------------------------------------------

def _tree_sizes(case):
    """Per sequence: new tokens, and tokens cached with them."""
    new = _between(case, "new", case["new"], (case["new"] + 1) // 2)
    total = _between(case, "len", case["length"], (case["length"] + 3) // 4)
    return new, [max(a, b) for a, b in zip(new, total)]


def _prepare_tree(s, case, g, seed):
    tpp, dt, n = s["tpp"], s["dt"], case["n_seq"]
    new, total = _tree_sizes(case)
    width = _pages(max(total), tpp)
    s.update(lens=_ints(total), starts=_ints(_sum_to(new)), T=sum(new), longest=max(total), nodes=max(new), width=width)
    there = torch.arange(width, device="cuda") < _ints([_pages(m, tpp) for m in total])[:, None]
    s["n_pages"] = int(2 * there.sum())
    table = torch.full((n, 2, width), -1, dtype=torch.int32, device="cuda")
    table[there[:, None, :].expand_as(table)] = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32)
    s["table"] = table
    s["pages"] = torch.empty((s["n_pages"], s["hidden"]), dtype=dt, device="cuda").normal_(generator=g)
    # twice the unit variance: logits of a few units, so that some tokens carry most of the weight
    s["q"] = torch.empty((s["T"], s["heads"] * s["dim"]), dtype=dt, device="cuda").normal_(generator=g) * 2
    words, parents, rows = _pages(s["nodes"], 64), _trees(new, seed), []
    for m in new:
        first = len(rows)
        for i in range(m):
            rows.append((rows[first + parents[first + i]] if i else 0) | 1 << i)
    s["bits"] = rows
    signed = [(r >> 64 * w & (2 ** 64 - 1)) for r in rows for w in range(words)]
    s["mask"] = _ints([x - 2 ** 64 if x >> 63 else x for x in signed], torch.int64).reshape(-1, words)
    _rows_of(s, new)


def _tree(s):
    if own:
        return s["pool"].kv_attend_tree(s["layout"], s["q"], s["table"], s["lens"], s["starts"], s["mask"], max_nodes=s["nodes"],
                                        scale=s["scale"], max_len=s["longest"])
    tpp, w, n, group = s["tpp"], s["kv"] * s["dim"], len(s["lens"]), s["heads"] // s["kv"]
    kv = s["pages"][s["table"].clamp(min=0).long()][..., : tpp * w].float()
    kv = kv.reshape(n, 2, -1, s["kv"], s["dim"])[:, :, : s["longest"]]
    t = torch.arange(kv.shape[2], device="cuda")
    there = t < s["lens"][:, None]
    kv = kv * there[:, None, :, None, None]
    k, v = kv[:, 0].transpose(1, 2).contiguous(), kv[:, 1].transpose(1, 2).contiguous()
    b, row = s["of"]
    m = s["most"]
    q = torch.zeros((n, m, s["kv"], group, s["dim"]), device="cuda")
    q[b, row] = s["q"].float().reshape(-1, s["kv"], group, s["dim"])
    q = q.permute(0, 2, 3, 1, 4).reshape(n, s["kv"], -1, s["dim"])          # rows: (head of the group, node)
    mask = torch.zeros((n, m, s["mask"].shape[1]), dtype=torch.int64, device="cuda")
    mask[b, row] = s["mask"]
    old = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1])
    node = t - old[:, None]                                                  # of each token; below 0: cached before
    j = node.clamp(0, 64 * mask.shape[2] - 1)
    word = mask.gather(2, (j // 64)[:, None].expand(n, m, -1))
    seen = there[:, None] & ((node < 0)[:, None] | ((word >> (j % 64)[:, None] & 1) > 0))
    x = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).unflatten(2, (group, -1))
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (group, -1)).permute(0, 3, 1, 2, 4)
    return o[b, row].reshape(s["T"], -1).to(s["dt"])


def _exact_tree(s):
    """Sequence by sequence and head by head, over its own pages alone."""
    kv, dim, tpp, group = s["kv"], s["dim"], s["tpp"], s["heads"] // s["kv"]
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    out = torch.zeros((s["T"], s["heads"], dim), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        first, m = starts[b], starts[b + 1] - starts[b]
        count = _pages(n, tpp)
        rows = s["pages"][s["table"][b, :, :count].reshape(-1).long(), : tpp * kv * dim]
        rows = rows.reshape(2, count * tpp, kv, dim)[:, :n].double()
        hidden = torch.tensor([[not s["bits"][first + i] >> j & 1 for j in range(m)] for i in range(m)], device="cuda")
        hidden = torch.cat([torch.zeros((m, n - m), dtype=torch.bool, device="cuda"), hidden], 1)
        for j in range(kv):
            for h in range(j * group, (j + 1) * group):
                q = s["q"][first: first + m, h * dim: (h + 1) * dim].double()
                x = (q @ rows[0, :, j].T) * s["scale"]
                out[first: first + m, h] = torch.softmax(x.masked_fill(hidden, -math.inf), dim=1) @ rows[1, :, j]
    return out.reshape(s["T"], -1)


# ---- keeping the accepted path ----------------------------------------------------------------------------------------

def _accept_sizes(case):
    """Per sequence: how deep its drafts are.  `chains` of them hang on the root, one behind the other."""
    return _between(case, "depth", case["depth"], 1)


def _walks(case, seed):
    """Per sequence: its parents, and how many tokens of which draft the model agrees with."""
    r = random.Random(seed)
    chains = case["chains"]
    for d in _accept_sizes(case):
        yield [0] + [1 + c * d + i - 1 if i else 0 for c in range(chains) for i in range(d)], r.randrange(chains), r.randint(0, d), d


def _prepare_accept(s, case, g, seed):
    tpp, layers, n, past, dt = s["tpp"], case["layers"], case["n_seq"], case["past"], s["dt"]
    r = random.Random(seed + 1)
    parents, tokens, targets, new = [], [], [], []
    for par, chain, agreed, d in _walks(case, seed):
        tok = [r.randrange(32000) for _ in par]
        tgt = [r.randrange(32000, 64000) for _ in par]       # tokens that nothing drafted
        node = 0
        for i in range(agreed):
            tgt[node], node = tok[1 + chain * d + i], 1 + chain * d + i
        parents += par
        tokens += tok
        targets += tgt
        new.append(len(par))
    total = [past + m for m in new]
    width, shared = _pages(max(total), tpp), past // tpp     # whole pages of a common prefix, held by all
    own_pages = [_pages(m, tpp) - shared for m in total]
    s["n_pages"] = 2 * layers * (shared + sum(own_pages))
    ids = torch.randperm(s["n_pages"], generator=g, device="cuda").to(torch.int32)
    table = torch.full((layers, n, 2, width), -1, dtype=torch.int32, device="cuda")
    table[..., :shared] = ids[: 2 * layers * shared].reshape(layers, 1, 2, shared)
    e = torch.arange(width, device="cuda")
    mine = (e >= shared) & (e < shared + _ints(own_pages)[:, None])
    table[mine[None, :, None, :].expand_as(table)] = ids[2 * layers * shared:]
    s["table"], s["pages"] = table, torch.empty((s["n_pages"], s["hidden"]), dtype=dt, device="cuda").normal_(generator=g)
    s.update(parents=_ints(parents), tokens=_ints(tokens), targets=_ints(targets), starts=_ints(_sum_to(new)), lens=_ints(total),
             nodes=1 + case["chains"] * case["depth"])
    _rows_of(s, new)
    z = dict(dtype=torch.int32, device="cuda")
    s["out"] = (torch.empty(n, **z), torch.empty((n, s["nodes"]), **z), torch.empty(n, **z), torch.empty(n, **z))


def _accept(s):
    if own:
        a = s["pool"].kv_accept(s["layout"], s["table"], s["lens"], s["starts"], s["tokens"], s["targets"], s["parents"], s["nodes"],
                                out=s["kept"])
        return [a.lens, a.path, a.n_path, a.next, s["pages"]]
    tpp, w, n, m = s["tpp"], s["kv"] * s["dim"], len(s["lens"]), s["most"]
    par, tok, tgt = _padded(s, s["parents"], -1), _padded(s, s["tokens"], -1), _padded(s, s["targets"], -2)
    par[:, 0] = -1
    j = torch.arange(m, device="cuda")
    fits = (par[:, None, :] == j[:, None]) & (tok[:, None, :] == tgt[:, :, None])      # [node][child]
    first = torch.where(fits, j, m).amin(-1)
    on = _closure(first[:, :, None] == j)[:, 0]                                         # what the root leads to
    count = on.sum(1)
    path = torch.where(on, j, m).sort(1).values
    path = torch.where(path < m, path, -1)
    last = path.gather(1, (count - 1)[:, None])
    old = s["lens"].long() - (s["starts"][1:] - s["starts"][:-1])
    b, i = (path >= 0).nonzero(as_tuple=True)
    src, dst = old[b] + path[b, i], old[b] + i
    held = s["pages"][:, : tpp * w].unflatten(1, (tpp, w))
    held[s["table"][:, b, :, dst // tpp].long(), (dst % tpp)[:, None, None]] = \
        held[s["table"][:, b, :, src // tpp].long(), (src % tpp)[:, None, None]]
    wide = torch.full((n, s["nodes"]), -1, dtype=torch.int32, device="cuda")
    wide[:, :m] = path
    return [(old + count).int(), wide, count.int(), tgt.gather(1, last)[:, 0].int(), s["pages"]]


def _exact_accept(s):
    """Walked on the host; the pages are moved, not computed: token by token, from what lay there before."""
    tpp, w = s["tpp"], s["kv"] * s["dim"]
    parents, tokens, targets = s["parents"].tolist(), s["tokens"].tolist(), s["targets"].tolist()
    starts, lens, table = s["starts"].tolist(), s["lens"].tolist(), s["table"].cpu().numpy()
    moved = []
    for b, n in enumerate(lens):
        first, m = starts[b], starts[b + 1] - starts[b]
        node, i = 0, 0
        while True:
            if node != i:
                a, z = n - m + node, n - m + i
                moved += [(int(x) * s["hidden"] + a % tpp * w, int(y) * s["hidden"] + z % tpp * w)
                          for x, y in zip(table[:, b, :, a // tpp].reshape(-1), table[:, b, :, z // tpp].reshape(-1))]
            to = [c for c in range(1, m) if parents[first + c] == node and tokens[first + c] == targets[first + node]]
            if not to:
                break
            node, i = to[0], i + 1
    before = s["pages"].reshape(-1)
    pages = s["pages"].double()
    at = torch.arange(w, device="cuda")
    for x in range(0, len(moved), 4096):
        pair = _ints(moved[x: x + 4096], torch.int64)
        pages.view(-1)[(pair[:, 1:] + at).reshape(-1)] = before[(pair[:, :1] + at).reshape(-1)].double()
    return [None, None, None, None, pages]


def work(case):
    """Each input read once, each output written once; products and sums of attention alone."""
    heads, kv, dim, hidden, tpp = GEOMETRY[case["geo"]]
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "plan":
        lens, new, held = _plan_sizes(case)
        moved = 0
        for n, m, h in zip(lens, new, held):
            want = _pages(n + m, tpp)
            moved += 4 * (want - n // tpp) + 4 * max(0, want - h) + 8 * max(0, h - want) + 8 * m    # entries, slots
        T, n = sum(new), case["n_seq"]
        words = _pages(case["new"], 64) if case["tree"] else 0
        return {"bytes": 2 * case["layers"] * moved + 4 * 7 * n + 4 * T + (4 + 8 * words) * T * case["tree"], "flops": 0}
    if case["op"] == "rope":
        T = case["T"]
        tables = min(T, case["far"]) * case["rot"] * 4
        return {"bytes": 2 * T * (heads + 2 * kv) * dim * size + 20 * T + tables, "flops": 3 * T * (heads + kv) * case["rot"]}
    if case["op"] == "tree":
        new, total = _tree_sizes(case)
        T, words = sum(new), _pages(max(new), 64)
        pairs = sum(m * (n - m) + 2 * m for m, n in zip(new, total))        # (row, token) pairs: at least two of the tree's
        pages = sum(_pages(n, tpp) for n in total)
        return {"bytes": 2 * sum(total) * kv * dim * size + 8 * pages + 2 * T * heads * dim * size + 8 * words * T,
                "flops": 4 * pairs * heads * dim}
    T = sum(1 + case["chains"] * d for d in _accept_sizes(case))
    c = case["chains"]
    moves = sum(d / 2 * (c - 1) / c for d in _accept_sizes(case))            # on average; the first draft lies in its place
    return {"bytes": 2 * moves * case["layers"] * 2 * kv * dim * size + 12 * T + 4 * case["n_seq"] * (5 + case["chains"] * case["depth"]),
            "flops": 0}
