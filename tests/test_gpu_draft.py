"""A step of drafted tokens on the device, call by call, against the plain forms in draft_ref.py.

Tolerances are its bounds on the float32 sums plus half a step of the output's type (bfloat16 2^-8, float32 2^-24,
relative); whole numbers are equal."""
import numpy as np
import pytest
import torch

import draft_ref
import kv_ref
import rank_gemm_unified_amd as rg
from gpu_helpers import say

pytestmark = pytest.mark.gpu

# heads, K/V heads, head dim, hidden, tokens a page
GEO = {
    "mha64": (4, 4, 64, 256, 1),
    "gqa64": (8, 2, 64, 256, 2),
    "mqa128": (4, 1, 128, 704, 5),         # five tokens a page, 64 elements unused
    "group16": (16, 1, 128, 128, 1),
    "group3": (6, 2, 128, 512, 2),
    "dim256": (4, 2, 256, 2048, 4),
    "mha128": (32, 32, 128, 4096, 1),
    "kv8": (32, 8, 128, 4096, 4),
}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(x, dtype=np.int32):
    return torch.as_tensor(np.asarray(x, dtype), device="cuda")


class Trees:
    """A pool full of random vectors, sequences with pages in random order, trees of new tokens at their ends."""

    def __init__(self, geo, dtype, lens, new, seed=1, gap=0, max_nodes=None, near=6, extra_pages=3, max_len=None):
        nh, nkv, dim, H, tpp = GEO[geo]
        self.layout, self.dt, self.lens, self.n = rg.lora_kv_layout_t(nh, nkv, dim, tpp), DT[dtype], list(lens), len(lens)
        rng = np.random.default_rng(seed)
        count = [-(-n // tpp) for n in lens]
        self.mp = max(1, max(count)) + extra_pages
        order = rng.permutation(2 * sum(count) + 7).astype(np.int32)
        self.table = np.full((self.n, 2, self.mp), -1, np.int32)
        at = 0
        for b, c in enumerate(count):
            for r in range(2):
                self.table[b, r, :c] = order[at:at + c]
                at += c
        self.pool = rg.Pool(len(order), H, rg.LORA_BF16 if self.dt is torch.bfloat16 else rg.LORA_F32, max_rank=1)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool.pages.normal_(generator=g)
        self.new, self.starts = list(new), [gap]
        for m in new:
            self.starts.append(self.starts[-1] + m)
        self.T = self.starts[-1] + gap
        self.nodes = max(1, max(new)) if max_nodes is None else max_nodes
        self.bits = [0] * gap + draft_ref.mask_rows(draft_ref.random_trees(rng, new, near), new) + [0] * gap
        self.q = torch.empty((self.T, nh * dim), dtype=self.dt, device="cuda").normal_(generator=g) * 1.5
        self.d_table, self.d_lens, self.d_start = dev(self.table), dev(self.lens), dev(self.starts)
        self.scale, self.max_len, self.rng = dim ** -0.5, max_len, rng

    def mask(self):
        return dev(draft_ref.mask_words(self.bits, (self.nodes + 63) // 64), np.int64)

    def run(self, **kw):
        args = dict(max_nodes=self.nodes, max_len=self.max_len)
        return self.pool.kv_attend_tree(self.layout, self.q, self.d_table, self.d_lens, self.d_start, self.mask(), **{**args, **kw})

    def ref(self):
        # bfloat16 weights in the product with V: two numbers, as one token's, up to 16 rows (nodes times query heads) of a
        # K/V head; of more rows rounded once, as a chunk's (kv_ref.ROUNDED).  float32 as they are
        rows = self.nodes * (self.layout.n_heads // self.layout.n_kv_heads)
        return draft_ref.attend(self.pool.pages, self.layout, self.q, self.table, self.lens, self.starts, self.bits, self.scale,
                                kv_ref.ROUNDED[self.dt, rows > 16])

    def errors(self):
        return rg.lora_check_device_errors(self.pool.handle, check=False)


def close(got, want, tol, dt, what):
    got = got.detach().to("cpu", torch.float64).numpy()
    rows = ~np.isnan(want)
    off, most = np.abs(got - want), tol * (1 + kv_ref.HALF[dt]) + kv_ref.HALF[dt] * np.abs(want) + 1e-30
    assert np.isfinite(got[rows]).all(), what
    say(f"{what}: worst error {np.max(np.where(rows, off / most, 0), initial=0):.3f} of the bound")
    assert not (rows & (off > most)).any(), (what, int((rows & (off > most)).sum()))


def check(c, what="tree"):
    want, tol = c.ref()
    close(c.run(), want, tol, c.dt, what)
    assert c.errors() == rg.LORA_OK


# ---- attention of trees ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", list(GEO))
def test_trees_on_mixed_caches(geo, dtype):
    check(Trees(geo, dtype, [40, 9, 131, 64, 1, 33], [9, 9, 3, 16, 1, 2]), geo)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("nodes", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 129, 255, 256])
def test_tree_sizes(nodes, dtype):
    """From one node, the decode step, to the largest tree: one to four words of mask, blocks that end inside a tree."""
    check(Trees("gqa64", dtype, [nodes, nodes + 1, nodes + 100], [nodes, max(1, nodes - 1), (nodes + 1) // 2]), f"{nodes} nodes")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", ["mha64", "mqa128", "group16", "dim256", "mha128"])
def test_long_caches_are_cut_into_ranges(geo, dtype):
    c = Trees(geo, dtype, [2500, 7, 1300, 0, 64], [5, 7, 13, 0, 2], seed=3)
    assert rg.lora_kv_attend_tree_workspace_size(c.pool.handle, c.layout, 5, 13, c.mp * c.layout.tokens_per_page) > 0
    check(c, geo)


def test_one_long_cache_on_every_workgroup():
    check(Trees("kv8", "bf16", [9001], [32], seed=5), "one cache of 9001 tokens")
    check(Trees("gqa64", "f32", [9001], [3], seed=6), "float32")


@pytest.mark.parametrize("offset", range(0, 33, 3))
def test_trees_that_begin_at_every_place_of_a_tile(offset):
    check(Trees("mha64", "bf16", [offset + 40, offset + 5], [40, 5], seed=offset), f"behind {offset}")
    check(Trees("dim256", "f32", [offset + 21], [21], seed=offset), f"float32 behind {offset}")


@pytest.mark.parametrize("max_len", [None, 5000])
def test_rows_outside_and_empty_sequences(max_len):
    """Rows behind the last sequence and before the first stay; a length of 0 is zero rows; a sequence without rows is
    skipped."""
    c = Trees("gqa64", "bf16", [50, 0, 20, 12], [5, 4, 0, 3], gap=3, extra_pages=2600, max_len=max_len)
    out = torch.full_like(c.q, 7.0)
    want, tol = c.ref()
    c.run(out=out)
    close(out, want, tol, c.dt, "padded")
    assert (out[:3] == 7).all() and (out[-3:] == 7).all() and (out[3 + 5: 3 + 9] == 0).all()
    assert c.errors() == rg.LORA_OK


def test_masks_of_any_kind():
    """No bit at all, bits of later nodes, not the row itself, bits behind the last node, every bit."""
    for old in (0, 7):
        c = Trees("gqa64", "bf16", [old + 6, old + 5], [6, 5], seed=9)
        c.bits = [0, 0b111110, 0b000100, 0, 1 << 5, 0b101010, 0, 0b1, 0b11110, 2 ** 64 - 1, 1 << 63 | 1]
        want, tol = c.ref()
        out = c.run()
        close(out, want, tol, c.dt, f"behind {old}")
        if old == 0:
            assert (out[0] == 0).all() and (out[3] == 0).all() and (out[6] == 0).all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("where", ["K", "V"])
def test_hidden_nodes_reach_no_row(where, dtype, value):
    """A node's K and V hold what is not finite: rows that do not see it come out as if it were not there; rows that see a
    value of it are not finite there."""
    c = Trees("gqa64", dtype, [45, 1100], [12, 20], seed=4)
    want, tol = c.ref()
    node, tpp = 5, c.layout.tokens_per_page
    for b in range(2):
        t = c.lens[b] - c.new[b] + node
        row = c.pool.pages[int(c.table[b, 0 if where == "K" else 1, t // tpp])]
        row[t % tpp * 128: t % tpp * 128 + 128] = value
    out = c.run()
    for b in range(2):
        rows = [c.starts[b] + i for i in range(c.new[b])]
        free = [r for r in rows if not c.bits[r] >> node & 1]
        seeing = [r for r in rows if c.bits[r] >> node & 1]
        assert free and seeing
        close(out[free], want[free], tol[free], c.dt, f"{where} {value}")
        if where == "V" or value != value:
            assert not torch.isfinite(out[seeing]).any()


def test_bad_pages_and_lengths_are_recorded():
    c = Trees("gqa64", "bf16", [50, 40, 30, 20], [5, 4, 3, 2], seed=2)
    c.table[0, 0, 3] = 10 ** 6
    c.table[1, 1, 2] = -5
    c.d_table = dev(c.table)
    want, tol = c.ref()
    close(c.run(), want, tol, c.dt, "bad pages hide their tokens")
    assert c.errors() == rg.LORA_EDEVICE
    for lens in ([50, -1, 30, 20], [50, 3, 30, 20], [50, 10 ** 6, 30, 20]):   # negative, below the rows, over the table
        c = Trees("gqa64", "bf16", [50, 40, 30, 20], [5, 4, 3, 2], seed=2)
        c.d_lens = dev(lens)
        c.lens[1] = 0
        want, tol = c.ref()
        close(c.run(), want, tol, c.dt, str(lens))
        assert c.errors() == rg.LORA_EDEVICE
    c = Trees("gqa64", "bf16", [50, 40, 30], [5, 14, 3], seed=2, max_nodes=8)   # more nodes than the call's most
    out = torch.full_like(c.q, 7.0)
    want, tol = c.ref()
    c.run(out=out)
    keep = np.r_[0:5, 19:22]
    close(out[keep], want[keep], tol[keep], c.dt, "others")
    assert (out[5:19] == 7).all() and c.errors() == rg.LORA_EDEVICE


@pytest.mark.parametrize("scale", [0.0, -0.3, 40.0])
def test_scales(scale):
    c = Trees("group3", "f32", [70, 33], [9, 4], seed=8)
    c.scale = scale
    want, tol = c.ref()
    close(c.run(scale=scale), want, tol, c.dt, f"scale {scale}")


def test_strided_rows_and_given_buffers():
    c = Trees("gqa64", "bf16", [50, 2100], [5, 11], seed=12)
    wide = torch.zeros((c.T, 3 * 512 + 64), dtype=c.dt, device="cuda")
    wide[:, 512:1024] = c.q
    res = torch.full((c.T, 1024), 3.0, dtype=c.dt, device="cuda")
    need = rg.lora_kv_attend_tree_workspace_size(c.pool.handle, c.layout, 2, c.nodes, c.mp * 2)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want, tol = c.ref()
    c.q = wide[:, 512:1024]
    c.run(out=res[:, :512], workspace=ws)
    close(res[:, :512], want, tol, c.dt, "strided")
    assert (res[:, 512:] == 3).all()


def test_repeats_bit_for_bit():
    c = Trees("kv8", "bf16", [3000, 1031, 77], [16, 9, 16], seed=14)
    first = c.run()
    for _ in range(3):
        assert torch.equal(first, c.run())


# ---- the plan -------------------------------------------------------------------------------------------------------

class Steps:
    def __init__(self, tpp, layers, lens, held, free, seed=0, max_pages=40, head=None):
        rng = np.random.default_rng(seed)
        self.layers, self.tpp, self.n = layers, tpp, len(lens)
        self.layout = rg.lora_kv_layout_t(2, 1, 64, tpp)
        groups = sum(max(0, h) for h in held) + free + 2
        ids = rng.permutation(2 * layers * groups).astype(np.int32).reshape(groups, layers, 2)
        self.pool = rg.Pool(2 * layers * groups, 64 * tpp, rg.LORA_BF16, max_rank=1)
        self.table = np.full((layers, self.n, 2, max_pages), -7, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[:, b, :, : max(0, h)] = ids[at:at + max(0, h)].transpose(1, 2, 0)
            at += max(0, h)
        self.head = int(rng.integers(groups)) if head is None else head
        self.stock = np.full((groups, layers, 2), -9, np.int32)
        for i in range(free):
            self.stock[(self.head + i) % groups] = ids[at + i]
        self.lens, self.held, self.state = list(lens), list(held), [self.head, free, 0, 0]
        self.num_pages = 2 * layers * groups

    def check(self, counts, T=None, parents=None, max_nodes=0, in_place=False, max_len=None, errors=False):
        T = sum(counts) if T is None else T
        cap = self.table.shape[-1] * self.tpp if max_len is None else max_len
        want = draft_ref.plan(self.layers, self.tpp, counts, self.lens, self.held, self.table, self.stock, self.state, T, cap, parents,
                              max_nodes, self.num_pages)
        table, stock, lens, held, state = dev(self.table), dev(self.stock), dev(self.lens), dev(self.held), dev(self.state)
        out = None
        if in_place:
            z = dict(dtype=torch.int32, device="cuda")
            out = rg.KvPlan(torch.empty(self.n, **z), torch.empty(self.n + 1, **z),
                            torch.empty((self.layers, 2, T), dtype=torch.int64, device="cuda"), torch.empty(T, **z),
                            None if parents is None else torch.empty((T, (max_nodes + 63) // 64), dtype=torch.int64, device="cuda"),
                            lens, held, state)
        got = self.pool.kv_plan(self.layout, dev(counts), lens, held, table, stock, state, T, max_len=max_len,
                                parents=None if parents is None else dev(parents), max_nodes=max_nodes, out=out)
        for name in ("step_lens", "q_start", "slots", "positions", "lens", "held", "state"):
            assert np.array_equal(getattr(got, name).cpu().numpy(), np.asarray(want[name])), name
        if parents is not None:
            assert np.array_equal(got.mask.cpu().numpy(), want["mask"].view(np.int64))
        assert np.array_equal(table.cpu().numpy(), want["table"]) and np.array_equal(stock.cpu().numpy(), want["stock"])
        assert (rg.lora_check_device_errors(self.pool.handle, check=False) == rg.LORA_EDEVICE) == errors == want["err"]
        self.table, self.stock, self.lens, self.held, self.state = want["table"], want["stock"], want["lens"], want["held"], want["state"][:2] + [0, 0]
        return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tpp", [1, 4, 7])
@pytest.mark.parametrize("layers", [1, 3, 40])
def test_plans_follow_one_another(layers, tpp, in_place):
    """Prompts, steps of one token, trees, rollbacks and requests that end, over a ring that goes round."""
    s = Steps(tpp, layers, [0, 0, 0, 0, 0], [0, 0, 0, 0, 0], 5 * 40 // tpp + 5, seed=layers, max_pages=80 // tpp + 2)
    rng = np.random.default_rng(7)
    s.check([30, 1, 0, 17, 8], in_place=in_place)
    for step in range(6):
        counts = [int(x) for x in rng.integers(1, 7, 5)]
        counts[step % 5] = 0
        s.check(counts, T=sum(counts) + step, parents=draft_ref.random_trees(rng, counts) + [0] * step, max_nodes=6, in_place=in_place)
        s.lens = [max(0, n - int(rng.integers(0, max(1, c)))) for n, c in zip(s.lens, counts)]    # some drafts were refused
        s.check([1 if n else 0 for n in s.lens], in_place=in_place)
        if step == 3:
            s.lens[0] = s.lens[3] = 0                                                             # two requests end
            s.check([0, 0, 2, 0, 0], in_place=in_place)
            s.check([25, 0, 0, 11, 0], in_place=in_place)


@pytest.mark.parametrize("free", [0, 1, 4, 5, 9, 10])
def test_too_few_pages_refuse_the_first_that_lacks_them_and_those_behind(free):
    s = Steps(2, 2, [3, 4, 10, 1, 6], [2, 2, 5, 4, 3], free)
    want = s.check([1, 7, 0, 2, 4])
    assert want["state"][2] == (0 if free >= 6 else 1 if free >= 4 else 2)


def test_a_stock_that_comes_from_elsewhere_is_recorded():
    for state in ([-1, 3, 0, 0], [0, 99, 0, 0], [500, 1, 0, 0]):
        s = Steps(2, 2, [3, 4], [2, 6], 3)
        s.state = state
        s.check([1, 3], errors=True)
    s = Steps(1, 1, [0, 2], [6, 2], 3, head=0)
    s.state[1] = len(s.stock) - 2                           # says it is nearly full: six pages cannot come back
    s.check([0, 0], T=0, errors=True)


@pytest.mark.parametrize("counts,lens,held,max_len", [
    ([3, -1, 2], [5, 5, 5], [3, 3, 3], None), ([3, 9, 2], [5, 5, 5], [3, 3, 3], 13), ([1, 1, 1], [5, -2, 5], [3, 3, 3], None),
    ([1, 1, 1], [5, 500, 5], [3, 3, 3], None), ([1, 1, 1], [5, 9, 5], [3, 4, 3], None), ([1, 1, 1], [5, 5, 5], [3, -4, 3], None),
    ([1, 1, 1], [5, 5, 5], [3, 41, 3], None), ([1 << 30, 1, 1], [5, 5, 5], [3, 3, 3], None)])
def test_bad_numbers_leave_a_sequence_as_it_is(counts, lens, held, max_len):
    s = Steps(2, 3, lens, [h if 0 <= h <= 40 else 3 for h in held], 30)
    s.held = list(held)
    s.check(counts, T=12, max_len=max_len, errors=True)


def test_rows_behind_the_last_and_bad_parents():
    s = Steps(2, 2, [5, 5, 5], [3, 3, 3], 30)
    s.check([4, 4, 4], T=9, errors=True)                    # the third has no room
    s = Steps(2, 2, [5, 5, 5], [3, 3, 3], 30)
    s.check([4, 4, 4], parents=[0, 0, 1, 3, 0, 0, -1, 2, 9, 0, 1, 2], max_nodes=4, errors=True)
    s = Steps(2, 2, [5, 5, 5], [3, 3, 3], 30)
    s.check([4, 5, 4], T=13, parents=[0] * 13, max_nodes=4, errors=True)
    s = Steps(2, 2, [5, 5], [3, 3], 30)
    s.stock[s.head] = 10 ** 6                               # a page outside the pool
    s.check([4, 4], errors=True)


@pytest.mark.parametrize("nodes", [63, 64, 65, 200, 256])
def test_masks_of_large_trees(nodes):
    rng = np.random.default_rng(nodes)
    for near in (1, 6, 256):                                # a chain, and wide trees
        s = Steps(8, 1, [3, 0, 17], [1, 0, 3], 120, max_pages=60)
        sizes = [nodes, nodes - 1, nodes // 2]
        s.check(sizes, parents=draft_ref.random_trees(rng, sizes, near), max_nodes=nodes)


def test_many_sequences_and_one_prompt_over_many_workgroups():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 30, 700)]
    s = Steps(4, 2, lens, [-(-n // 4) + int(rng.integers(0, 2)) for n in lens], 900, max_pages=12)
    s.check([int(x) for x in rng.integers(0, 4, 700)], T=1200, in_place=True)
    s.lens = [0 if b % 3 else n for b, n in enumerate(s.lens)]
    s.check([0] * 700, T=0, in_place=True)
    s = Steps(1, 2, [5, 0, 9], [5, 0, 9], 3000, max_pages=2600)
    s.check([1, 2500, 3], in_place=True)


# ---- rotary write ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo,rot", [("mha64", 64), ("mha64", 16), ("gqa64", 48), ("mqa128", 128), ("dim256", 256), ("dim256", 80), ("mha128", 128)])
@pytest.mark.parametrize("T,in_place", [(1, False), (70, True), (1500, False)])
def test_rope(geo, rot, dtype, pairs, T, in_place):
    nh, nkv, dim, H, tpp = GEO[geo]
    lay, dt, rng = rg.lora_kv_layout_t(nh, nkv, dim, tpp), DT[dtype], np.random.default_rng(T)
    pool = rg.Pool(2 * T + 5, H, rg.LORA_BF16 if dtype == "bf16" else rg.LORA_F32, max_rank=1)
    g = torch.Generator(device="cuda").manual_seed(T)
    pool.pages.normal_(generator=g)
    before = pool.pages.clone()
    rope = rg.Rope.of(5000, rot, interleaved=pairs)
    rows = torch.empty((T, (nh + 2 * nkv) * dim + 8), dtype=dt, device="cuda").normal_(generator=g)
    q, k, v = rows[:, : nh * dim], rows[:, nh * dim: (nh + nkv) * dim], rows[:, (nh + nkv) * dim: (nh + 2 * nkv) * dim]
    host = [x.double().cpu().numpy() for x in (q, k, v)]
    slots = rng.permutation((2 * T + 5) * tpp)[: 2 * T].reshape(2, T)
    pos = rng.integers(0, 5000, T)
    skip = rng.random(T) < 0.2
    slots[:, skip] = -1
    q_out = q if in_place else torch.full((T, nh * dim), 5.0, dtype=dt, device="cuda")
    want_q = q_out.double().cpu().numpy()
    got = pool.kv_write_rope(lay, rope, q, k, v, dev(slots, np.int64), dev(pos), q_out=q_out)
    assert got is q_out and rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_OK
    table = rope.table.double().cpu().numpy()
    tq, eq = draft_ref.rope(host[0], table, pos, nh, dim, pairs)
    tk, ek = draft_ref.rope(host[1], table, pos, nkv, dim, pairs)
    want_q[~skip] = tq[~skip]
    close(got, want_q, np.where(skip[:, None], 0, eq), dt, "q")
    want, tol = before.double().cpu().numpy(), np.zeros(before.shape)
    w = nkv * dim
    for t in range(T):
        if not skip[t]:
            a, b = slots[0, t], slots[1, t]
            want[a // tpp, a % tpp * w: a % tpp * w + w], tol[a // tpp, a % tpp * w: a % tpp * w + w] = tk[t], ek[t]
            want[b // tpp, b % tpp * w: b % tpp * w + w] = host[2][t]
    close(pool.pages, want, tol, dt, "pages")
    same = torch.as_tensor(tol == 0, device="cuda")
    assert torch.equal(torch.where(same, pool.pages.double(), 0.0), torch.where(same, torch.as_tensor(want, device="cuda"), 0.0))


def test_rope_keys_alone_and_bad_rows():
    nh, nkv, dim, H, tpp = GEO["gqa64"]
    lay = rg.lora_kv_layout_t(nh, nkv, dim, tpp)
    pool = rg.Pool(20, H, rg.LORA_F32, max_rank=1)
    pool.pages.zero_()
    rope = rg.Rope.of(7, 64)
    k = torch.randn((6, 128), device="cuda")
    q, q_out = torch.randn((6, 512), device="cuda"), torch.full((6, 512), 9.0, device="cuda")
    slots = dev([[0, 2, 40, 4, -1, 6], [1, 3, 5, -1, 7, 9]], np.int64)
    pool.kv_write_rope(lay, rope, q, k, k, slots, dev([0, 6, 1, 1, 1, 7]), q_out=q_out)
    assert rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_EDEVICE
    assert (q_out[2:] == 9).all() and (q_out[:2] != 9).all()
    held = pool.pages.view(40, 128)
    assert torch.equal(held[1], k[0]) and torch.equal(held[3], k[1]) and (held[4:] == 0).all()
    assert torch.equal(held[0], k[0])                       # position 0 turns nothing
    pool.pages.zero_()
    assert pool.kv_write_rope(lay, rope, None, k[:2], k[:2], dev([[0, 2], [1, 3]], np.int64), dev([0, 0])) is None
    assert torch.equal(held[:4], k[:2].repeat_interleave(2, 0))


# ---- acceptance -----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", ["mha64", "gqa64", "mqa128", "dim256", "mha128"])
@pytest.mark.parametrize("near,most", [(1, 40), (3, 30), (8, 256)])
def test_accepted_paths(geo, dtype, near, most):
    nh, nkv, dim, H, tpp = GEO[geo]
    lay, layers, rng = rg.lora_kv_layout_t(nh, nkv, dim, tpp), 3, np.random.default_rng(most)
    new = [1, most, 0, most // 2, 5, 3]
    old = [3, 0, 9, 17, 64, 2]
    lens = [o + m for o, m in zip(old, new)]
    lens[5] = 0                                             # refused by the plan: rows, but no step
    starts = np.concatenate([[2], 2 + np.cumsum(new)])
    T = int(starts[-1]) + 3
    parents = [0, 0] + draft_ref.random_trees(rng, new, near) + [0] * 3
    tokens = [int(x) for x in rng.integers(0, 2 if near > 1 else 1, T)]      # few tokens: paths go deep, and choose
    targets = [int(x) for x in rng.integers(0, 2 if near > 1 else 1, T)]
    mp = -(-max(lens) // tpp) + 1
    order = rng.permutation(2 * layers * 6 * mp).astype(np.int32)
    table = order.reshape(layers, 6, 2, mp)
    pool = rg.Pool(len(order), H, rg.LORA_BF16 if dtype == "bf16" else rg.LORA_F32, max_rank=1)
    pool.pages.normal_(generator=torch.Generator(device="cuda").manual_seed(most))
    want = pool.pages.clone()
    z = dict(dtype=torch.int32, device="cuda")
    out = rg.KvAccepted(torch.full((6,), 77, **z), torch.full((6, most), 77, **z), torch.full((6,), 77, **z), torch.full((6,), 77, **z))
    got = pool.kv_accept(lay, dev(table), dev(lens), dev(starts), dev(tokens), dev(targets), dev(parents), most, out=out)
    w = nkv * dim
    for b in range(6):
        m = new[b] if lens[b] else 0
        path = draft_ref.accept(parents, tokens, targets, m, int(starts[b]))
        assert int(got.n_path[b]) == len(path) and got.path[b].tolist() == path + [-1] * (most - len(path))
        assert int(got.lens[b]) == (old[b] + len(path) if m else 77)
        assert int(got.next[b]) == (targets[int(starts[b]) + path[-1]] if m else -1)
        for i, node in enumerate(path):
            a, z_ = old[b] + node, old[b] + i
            for l in range(layers):
                for r in range(2):
                    want[int(table[l, b, r, z_ // tpp]), z_ % tpp * w: z_ % tpp * w + w] = \
                        want[int(table[l, b, r, a // tpp]), a % tpp * w: a % tpp * w + w].clone()
    assert torch.equal(pool.pages, want) and rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_OK


def test_acceptance_of_bad_numbers():
    nh, nkv, dim, H, tpp = GEO["gqa64"]
    lay = rg.lora_kv_layout_t(nh, nkv, dim, tpp)
    pool = rg.Pool(64, H, rg.LORA_F32, max_rank=1)
    pool.pages.normal_()
    before = pool.pages.clone()
    table = np.arange(64, dtype=np.int32).reshape(1, 4, 2, 8)
    table[0, 1, 0, 1] = 900                                 # place 3 of sequence 1, where node 2 would go from
    new, parents = [3, 4, 9, 2], [0, 0, -1, 0, 0, 0, 2, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1]
    starts = np.concatenate([[0], np.cumsum(new)])
    got = pool.kv_accept(lay, dev(table), dev([3, 4, 9, 1]), dev(starts), dev([1] * 18), dev([1] * 18), dev(parents), 8)
    assert rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_EDEVICE
    # node 2's parent is none; a tree of nine is over the most; a length below the rows counts as 0
    assert got.n_path.tolist() == [2, 2, 0, 0] and got.next.tolist() == [1, 1, -1, -1] and got.lens.tolist() == [2, 2, 9, 1]
    assert torch.equal(pool.pages, before)
