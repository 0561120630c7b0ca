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


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("geo,lens,new", [
    ("gqa64", [11 + b % 60 for b in range(512)], [5 + b % 2 for b in range(512)]),           # two heads a workgroup, sequences whole
    ("kv8", [1990, 2000, 1000, 30, 17, 700, 900, 1600], [16, 9, 16, 9, 16, 13, 10, 16]),     # and in ranges
    ("mha128", [700, 41, 90], [9, 16, 12]), ("mha64", [1300, 64], [30, 20])])
def test_a_node_of_one_key_head_reaches_its_rows_alone(geo, lens, new, value):
    """V of one node of one K/V head of each sequence is not finite: rows that see the node are not there, and nowhere else."""
    c = Trees(geo, "bf16", lens, new, seed=len(lens))
    want, tol = c.ref()
    dim, nkv, tpp = c.layout.head_dim, c.layout.n_kv_heads, c.layout.tokens_per_page
    wide = c.layout.n_heads // nkv * dim                    # columns of a K/V head's query heads
    clean = np.ones(want.shape, bool)
    for b in range(0, c.n, 3):
        node, kvh = 2 + b % 3, b % nkv
        t = c.lens[b] - c.new[b] + node
        at = (t % tpp * nkv + kvh) * dim
        c.pool.pages[int(c.table[b, 1, t // tpp]), at: at + dim] = value
        for i in range(c.new[b]):
            if c.bits[c.starts[b] + i] >> node & 1:
                clean[c.starts[b] + i, kvh * wide: (kvh + 1) * wide] = False
    out = c.run()
    dirty = torch.as_tensor(~clean, device="cuda")
    assert dirty.any() and not torch.isfinite(out[dirty]).any()
    close(torch.where(dirty, 0.0, out), np.where(clean, want, 0), np.where(clean, tol, 0), c.dt, geo)
    assert c.errors() == rg.LORA_OK


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


def test_paths_of_a_step_without_rows_are_empty():
    lay = rg.lora_kv_layout_t(8, 2, 64, 2)
    pool = rg.Pool(64, 256, rg.LORA_F32, max_rank=1)
    none = dev([])
    got = pool.kv_accept(lay, dev(np.arange(16).reshape(1, 2, 2, 4)), dev([0, 3]), dev([0, 0, 0]), none, none, none, 3)
    assert got.path.tolist() == [[-1] * 3] * 2 and got.n_path.tolist() == [0, 0] and got.next.tolist() == [-1, -1] and got.lens.tolist() == [0, 3]


# ---- every form of the attention, its limits ------------------------------------------------------------------------

# Rows of a K/V head: up to 16 by the first kernel in one block (float32 up to 32 in two, except for heads of 256), more by the
# other; heads a workgroup 4, 2, 1 and 2 (17 to 64 rows of bfloat16 and enough tokens), 1; whole sequences or ranges; pieces joined by
# sequences or by the places between ranges, one thread or all of a workgroup to a row.
@pytest.mark.parametrize("geo,dtype,lens,new", [
    ("mha64", "bf16", [1500, 1100], [3, 16]), ("mqa128", "bf16", [2100], [4]), ("gqa64", "bf16", [1300], [4]),
    ("mha64", "f32", [1200, 1030], [17, 32]), ("mqa128", "f32", [1100], [8]), ("gqa64", "f32", [1300, 64], [5, 8]),
    ("dim256", "f32", [700, 1100], [16, 9]), ("kv8", "bf16", [1990, 2000, 1000, 30, 1, 700, 900, 1600], [16, 5, 9, 16, 1, 3, 2, 16]),
    ("mha128", "bf16", [700, 1010, 33, 900], [17, 40, 33, 64]), ("mha128", "f32", [600, 33], [20, 33]),
    ("gqa64", "bf16", [200] * 40, [2] * 40), ("mha64", "bf16", [40 + b % 90 for b in range(150)], [b % 4 for b in range(150)]),
    ("kv8", "bf16", [5000], [64]), ("dim256", "bf16", [3000], [64]), ("kv8", "bf16", [30 + b % 50 for b in range(140)], [1 + b % 4 for b in range(140)]),
    ("mha128", "f32", [300 - 7 * b for b in range(18)], [33 - b for b in range(18)]), ("mha128", "bf16", [20 + b for b in range(32)], [20 - b % 5 for b in range(32)]),
    ("gqa64", "bf16", [5 + b % 90 for b in range(512)], [b % 6 for b in range(512)]), ("dim256", "bf16", [9 + b % 70 for b in range(512)], [b % 10 for b in range(512)]),
    ("gqa64", "f32", [9 + b % 60 for b in range(260)], [b % 10 for b in range(260)])],
    ids=lambda x: x if isinstance(x, str) else f"{len(x)}x{max(x)}")
def test_every_form(geo, dtype, lens, new):
    check(Trees(geo, dtype, lens, new, seed=len(lens)), geo)


def test_sequences_that_are_all_empty():
    for geo, dtype, nodes in (("mha64", "bf16", 4), ("mha64", "f32", 20), ("mha64", "bf16", 40)):
        for pages in (1, 4000):                             # whole sequences at a time, and in ranges
            c = Trees(geo, dtype, [0, 0, 0], [nodes, 1, 2], extra_pages=pages)
            out = c.run(out=torch.full_like(c.q, 7.0))
            assert (out == 0).all() and c.errors() == rg.LORA_OK
            c.d_start, c.nodes = dev([0, 0, 0, 0]), nodes
            assert (c.run(out=torch.full_like(c.q, 7.0)) == 7).all() and c.errors() == rg.LORA_OK


def test_the_most_sequences_and_heads():
    """65535 sequences of a token each: the output is that token's V.  1024 heads on one and 1024 on their own."""
    n = rg.LORA_MAX_SEQS
    lay = rg.lora_kv_layout_t(1, 1, 64, 1)
    pool = rg.Pool(2 * n, 64, rg.LORA_F32, max_rank=1)
    pool.pages.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    z = dict(dtype=torch.int32, device="cuda")
    stock = torch.randperm(2 * n, generator=torch.Generator().manual_seed(2)).int().view(n, 1, 2).cuda()
    table, one, none = torch.full((1, n, 2, 1), -1, **z), torch.ones(n, **z), torch.zeros(n, **z)
    plan = pool.kv_plan(lay, one, none, none, table, stock, dev([5, n, 0, 0]), n, parents=none, max_nodes=1)
    ring = torch.roll(stock, -5, 0)
    assert torch.equal(table.view(n, 2), ring.view(n, 2)) and plan.state.tolist() == [5, 0, 0, 0]
    assert torch.equal(plan.slots[0].t(), ring.view(n, 2).long()) and torch.equal(plan.q_start, torch.arange(n + 1, **z))
    out = pool.kv_attend_tree(lay, torch.randn((n, 64), device="cuda"), table[0], plan.step_lens, plan.q_start, plan.mask, 1)
    assert torch.equal(out, pool.pages[ring[:, 0, 1].long()])
    kept = pool.kv_accept(lay, table, plan.step_lens, plan.q_start, one, one, none, 1)
    assert (kept.n_path == 1).all() and (kept.lens == 1).all() and rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_OK
    for kv in (1, 1024):
        lay = rg.lora_kv_layout_t(1024, kv, 64, 1)
        pool = rg.Pool(100, 64 * kv, rg.LORA_BF16, max_rank=1)
        pool.pages.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
        q = torch.randn((2, 65536), device="cuda").bfloat16()
        bits, lens = [1, 3], [40]
        table = np.arange(100, dtype=np.int32).reshape(1, 2, 50)
        want, tol = draft_ref.attend(pool.pages, lay, q, table, lens, [0, 2], bits, 0.125, kv_ref.ROUNDED[torch.bfloat16, kv == 1])
        close(pool.kv_attend_tree(lay, q, dev(table), dev(lens), dev([0, 2]), dev([[b] for b in bits], np.int64), 2), want, tol,
              torch.bfloat16, f"1024 heads on {kv}")


@pytest.mark.parametrize("dtype", list(DT))
def test_pages_behind_four_gib(dtype):
    """A pool of more than 2^32 bytes whose sequences' pages are its last ones: written, read and moved there."""
    H, many = 4096, (1 << 32) // (4096 * (2 if dtype == "bf16" else 4)) + 300
    lay, dt = rg.lora_kv_layout_t(4, 2, 64, 32), DT[dtype]
    pool = rg.Pool(many, H, rg.LORA_BF16 if dtype == "bf16" else rg.LORA_F32, max_rank=1)
    last = pool.pages[-300:]
    last.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    small = rg.Pool(300, H, rg.LORA_BF16 if dtype == "bf16" else rg.LORA_F32, max_rank=1)
    small.pages.copy_(last)
    table = np.random.default_rng(1).permutation(300)[:2 * 2 * 70].reshape(1, 2, 2, 70).astype(np.int32)
    rope, g = rg.Rope.of(3000, 64), torch.Generator(device="cuda").manual_seed(2)
    for m in (5, 40):
        T, old = 2 * m, (2000, 61)
        q, k, v = (torch.randn((T, w), generator=g, device="cuda").to(dt) for w in (256, 128, 128))
        pos = np.concatenate([o + np.arange(m) for o in old])
        seq = np.arange(T) // m
        bits = draft_ref.mask_rows(draft_ref.random_trees(np.random.default_rng(m), [m, m]), [m, m])
        got = []
        for of, at in ((pool, many - 300), (small, 0)):
            tab = table + at
            slots = np.stack([tab[0, seq, r, pos // 32].astype(np.int64) * 32 + pos % 32 for r in range(2)])
            turned = of.kv_write_rope(lay, rope, q, k, v, dev(slots, np.int64), dev(pos))
            lens, start = dev([o + m for o in old]), dev([0, m, 2 * m])
            out = of.kv_attend_tree(lay, turned, dev(tab[0]), lens, start, dev([[b] for b in bits], np.int64), m)
            of.kv_accept(lay, dev(tab), lens, start, dev([1] * T), dev([1] * T), dev(draft_ref.random_trees(np.random.default_rng(m), [m, m])), m)
            assert rg.lora_check_device_errors(of.handle, check=False) == rg.LORA_OK
            got += [out, of.pages[-300:]]
        assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


# ---- streams, graphs and refusals -----------------------------------------------------------------------------------

class Step:
    """A step of the four calls over one pool, one layer, into given buffers, whose numbers can be drawn anew."""

    def __init__(self, max_pages, most=20):
        self.most = most
        self.layout, self.n, self.T, groups = rg.lora_kv_layout_t(8, 2, 64, 2), 3, 64, 3000
        self.pool = rg.Pool(2 * groups, 256, rg.LORA_BF16, max_rank=1)
        self.pool.pages.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
        z = dict(dtype=torch.int32, device="cuda")
        new = lambda *s: torch.zeros(s, **z)  # noqa: E731
        n, T = self.n, self.T
        self.table, self.stock = new(1, n, 2, max_pages), torch.randperm(2 * groups, generator=torch.Generator().manual_seed(4)).int().view(-1, 1, 2).cuda()
        self.buffers = [new(n), new(n), new(n), self.table, self.stock, dev([0, groups, 0, 0]), new(T)] + \
            [torch.zeros((T, w), dtype=torch.bfloat16, device="cuda") for w in (512, 128, 128)] + [new(T), new(T)]
        self.plan = rg.KvPlan(new(n), new(n + 1), torch.zeros((1, 2, T), dtype=torch.int64, device="cuda"), new(T),
                              torch.zeros((T, 1), dtype=torch.int64, device="cuda"), self.buffers[1], self.buffers[2], self.buffers[5])
        self.kept = rg.KvAccepted(self.buffers[1], new(n, most), new(n), new(n))

    def draw(self, seed):
        most = self.most
        rng, g = np.random.default_rng(seed), torch.Generator(device="cuda").manual_seed(seed)
        counts = [int(x) for x in rng.integers(1, most, self.n)]
        counts[seed % self.n] = 0 if seed % 2 else most
        parents = draft_ref.random_trees(rng, counts)
        self.buffers[0].copy_(dev(counts))
        self.buffers[6].copy_(dev(parents + [0] * (self.T - len(parents))))
        for t in self.buffers[7:10]:
            t.normal_(generator=g)
        for t in self.buffers[10:]:
            t.copy_(dev(rng.integers(0, 2, self.T)))

    def all(self):
        return [self.pool.pages, *self.buffers[1:6], *[t for t in self.plan if t is not None], *self.kept]

    def run(self, rope, **kw):
        counts, lens, held, table, stock, state, parents, q, k, v, tokens, targets = self.buffers
        pool, lay, plan, most = self.pool, self.layout, self.plan, self.most
        pool.kv_plan(lay, counts, lens, held, table, stock, state, self.T, parents=parents, max_nodes=most, out=plan, **kw)
        turned = pool.kv_write_rope(lay, rope, q, k, v, plan.slots[0], plan.positions, **kw)
        out = pool.kv_attend_tree(lay, turned, table[0], plan.step_lens, plan.q_start, plan.mask, most, **kw)
        pool.kv_accept(lay, table, plan.step_lens, plan.q_start, tokens, targets, parents, most, out=self.kept, **kw)
        return out


@pytest.mark.parametrize("max_pages,most", [(100, 4), (900, 4), (100, 20), (900, 20)])       # sequences whole, and in ranges
def test_captured_calls_replayed(max_pages, most):
    """One graph of the four calls, replayed with new numbers, beside the same calls run eagerly on a pool of the same contents."""
    rope, two = rg.Rope.of(2000, 64), [Step(max_pages, most), Step(max_pages, most)]
    start = [t.clone() for t in two[0].all()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two[0].draw(0)
        two[0].run(rope)
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip(two[0].all(), start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = two[0].run(rope)
    for t, s in zip(two[0].all(), start):
        assert torch.equal(t, s)                            # nothing ran yet
    for seed in range(8):
        for s in two:
            s.draw(seed)
        graph.replay()
        eager = two[1].run(rope)
        torch.randn(1000, device="cuda").sum().item()
        rows = int(two[1].plan.q_start[-1])
        assert torch.equal(out[:rows], eager[:rows]) and all(torch.equal(a, b) for a, b in zip(two[0].all(), two[1].all())), seed
    for s in two:
        assert rg.lora_check_device_errors(s.pool.handle, check=False) == rg.LORA_OK


@pytest.mark.parametrize("kind", ["stream", "handle", "default", "zero"])
def test_calls_on_a_given_stream(kind):
    rope, here, there = rg.Rope.of(2000, 64), Step(900), Step(900)
    stream = torch.cuda.Stream() if kind in ("stream", "handle") else torch.cuda.default_stream()
    other = torch.cuda.Stream()
    given = {"stream": stream, "handle": stream.cuda_stream, "default": stream, "zero": 0}[kind]
    for seed in range(3):
        here.draw(seed)
        there.draw(seed)
        want = here.run(rope)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):                      # the current one is not the call's
            got = there.run(rope, stream=given)
        torch.cuda.synchronize()
        rows = int(here.plan.q_start[-1])
        assert torch.equal(got[:rows], want[:rows]) and all(torch.equal(a, b) for a, b in zip(here.all(), there.all()))
    with torch.cuda.stream(other):                          # into new tensors
        b = there.buffers
        p = there.pool.kv_plan(there.layout, b[0], b[1], b[2], b[3], b[4], b[5], there.T, parents=b[6], max_nodes=20, stream=given)
        kept = there.pool.kv_accept(there.layout, b[3], p.step_lens, p.q_start, b[10], b[11], b[6], 20, stream=given)
    torch.cuda.synchronize()
    resting = b[0] == 0
    assert torch.equal(kept.lens[resting], p.step_lens[resting]) and (kept.n_path[~resting] > 0).all()


def test_arguments_refused():
    s, rope = Step(100), rg.Rope.of(50, 64)
    c, counts, lens, held, table, stock, state, parents, q, k, v, tokens, targets = s.pool, *s.buffers
    plan = lambda **kw: c.kv_plan(**{**dict(layout=s.layout, counts=counts, lens=lens, held=held, table=table, stock=stock, state=state,  # noqa: E731
                                            T=s.T, parents=parents, max_nodes=20), **kw})
    p = plan()
    write = lambda **kw: c.kv_write_rope(**{**dict(layout=s.layout, rope=rope, q=q, k=k, v=v, slots=p.slots[0], positions=p.positions), **kw})  # noqa: E731
    tree = lambda **kw: c.kv_attend_tree(**{**dict(layout=s.layout, q=q, table=table[0], lens=p.step_lens, q_start=p.q_start, mask=p.mask,  # noqa: E731
                                                   max_nodes=20), **kw})
    keep = lambda **kw: c.kv_accept(**{**dict(layout=s.layout, table=table, lens=p.step_lens, q_start=p.q_start, tokens=tokens, targets=targets,  # noqa: E731
                                              parents=parents, max_nodes=20), **kw})
    bad = [(plan, dict(counts=counts.long())), (plan, dict(counts=counts.cpu())), (plan, dict(lens=lens[:2])), (plan, dict(held=held.float())),
           (plan, dict(table=table[:, :, :, ::2])), (plan, dict(stock=stock[:, :, :1])), (plan, dict(state=state[:3])), (plan, dict(T=5)),
           (plan, dict(parents=parents[::2])), (plan, dict(out=s.plan, T=63, parents=parents[:63])), (plan, dict(out=s.plan, parents=None)),
           (plan, dict(out=s.plan, max_nodes=65)), (plan, dict(out=s.plan._replace(mask=None))),
           (write, dict(q=q.float())), (write, dict(k=k[:, :64])), (write, dict(v=v[1:])), (write, dict(slots=p.slots[0].int())),
           (write, dict(slots=p.slots[0, :, :9])), (write, dict(positions=p.positions.cpu())), (write, dict(q=None, q_out=q)),
           (write, dict(q_out=q[:9])), (write, dict(q_out=q.t())), (tree, dict(q=q.float())), (tree, dict(q=q[:, :256])),
           (tree, dict(table=table)), (tree, dict(lens=p.step_lens[:2])), (tree, dict(q_start=p.q_start[:3])), (tree, dict(mask=p.mask.int())),
           (tree, dict(mask=p.mask[:9])), (tree, dict(max_nodes=65)), (tree, dict(out=q[:9])), (tree, dict(out=q.cpu())),
           (tree, dict(workspace=torch.empty(9))), (keep, dict(tokens=tokens.long())), (keep, dict(targets=targets[:9])),
           (keep, dict(parents=parents.cpu())), (keep, dict(table=table[0])), (keep, dict(lens=held[:1])), (keep, dict(out=s.kept, max_nodes=19))]
    for i, (call, change) in enumerate(bad):
        with pytest.raises((ValueError, IndexError)):
            call(**change)
            print("taken:", i, list(change))
    for call, change in ((plan, dict(max_nodes=0)), (plan, dict(max_len=300)), (write, dict(q_out=q[:, :], k=q[:, :128])), (tree, dict(max_len=0)),
                         (tree, dict(scale=float("nan"))), (tree, dict(out=q)), (keep, dict(max_nodes=0))):
        with pytest.raises((rg.LoraError, ValueError)):
            call(**change)
            print("taken:", list(change))
    z = dict(dtype=torch.int32, device="cuda")
    for make in (lambda: rg.KvAccepted(*[torch.zeros(3, **z)] * 4), lambda: s.plan._replace(positions=torch.zeros(9, **z)),
                 lambda: rg.KvPlan(*s.plan[:7], torch.zeros(4, dtype=torch.int32)), lambda: rg.Rope(torch.zeros((5, 8, 2))),
                 lambda: rg.Rope(torch.zeros((5, 8, 2), device="cuda").double()), lambda: rg.Rope(torch.zeros((5, 7, 2), device="cuda")),
                 lambda: rg.Rope(torch.zeros((0, 8, 2), device="cuda"))):
        with pytest.raises(ValueError):
            make()
    assert rg.lora_check_device_errors(c.handle, check=False) == rg.LORA_OK
