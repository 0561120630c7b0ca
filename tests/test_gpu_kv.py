"""The KV-cache calls on the device, against plain float64 forms (kv_ref.py).

Tolerances are kv_ref's bounds on the float32 sums plus half a step of the output's type
(bfloat16 2^-8, float32 2^-24, relative)."""
import numpy as np
import pytest
import torch

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
    "group20": (40, 2, 64, 128, 1),        # more heads on a K/V head than a matrix tile has columns
    "group3": (6, 2, 128, 512, 2),
    "dim256": (4, 2, 256, 2048, 4),
    "mha128": (32, 32, 128, 4096, 1),
}
# so many heads that a prompt's query tiles are taken in pairs
WIDE = {
    "wide64": (256, 256, 64, 16384, 1),
    "wide64_kv64": (256, 64, 64, 4096, 1),
    "wide64_kv128": (256, 128, 64, 16384, 2),
    "wide128": (128, 128, 128, 16384, 1),
    "wide128_kv32": (128, 32, 128, 4096, 1),
}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Case:
    """A pool full of random vectors (every page, used or not), sequences with pages in random order."""

    def __init__(self, geo, dtype, lens, new=None, seed=1, extra_pages=3, gap=0):
        nh, nkv, dim, H, tpp = {**GEO, **WIDE}[geo]
        self.layout, self.dt = rg.lora_kv_layout_t(nh, nkv, dim, tpp), DT[dtype]
        self.lens, self.n = list(lens), len(lens)
        self.mp = max(1, max(-(-n // tpp) for n in lens)) + extra_pages
        rng = np.random.default_rng(seed)
        count = [-(-n // tpp) for n in lens]
        total = 2 * sum(count) + 7
        order = rng.permutation(total).astype(np.int32)
        self.table = np.full((self.n, 2, self.mp), -1, np.int32)
        at = 0
        for b, c in enumerate(count):
            for r in range(2):
                self.table[b, r, :c] = order[at:at + c]
                at += c
        self.pool = rg.Pool(total, H, rg.LORA_BF16 if self.dt is torch.bfloat16 else rg.LORA_F32, max_rank=1)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool.pages.normal_(generator=g)
        self.q_start = None
        self.T = self.n
        if new is not None:
            starts = [gap]
            for m in new:
                starts.append(starts[-1] + m)
            self.q_start, self.T = starts, starts[-1] + gap
        self.width = nh * dim
        self.q = (torch.empty((self.T, self.width), dtype=self.dt, device="cuda").normal_(generator=g) * 1.5)
        self.d_table, self.d_lens = self.dev(self.table), self.dev(self.lens)
        self.d_start = None if new is None else self.dev(self.q_start)
        self.cap = self.mp * tpp
        self.scale = dim ** -0.5
        self.g = g

    @staticmethod
    def dev(x):
        return torch.as_tensor(np.asarray(x, np.int32), device="cuda")

    def run(self, scores=None, prior=None, q=None, out=None, **kw):
        q = self.q if q is None else q
        if self.q_start is None:
            return self.pool.kv_attend(self.layout, q, self.d_table, self.d_lens, scores=scores, prior=prior, out=out, **kw)
        return self.pool.kv_attend_chunk(self.layout, q, self.d_table, self.d_lens, self.d_start, scores=scores,
                                         prior=prior, out=out, **kw)

    def ref(self):
        return kv_ref.attend(self.pool.pages, self.layout, self.q, self.table, self.lens, self.q_start, self.scale,
                             kv_ref.ROUNDED[self.dt, self.q_start is not None])

    def errors(self):
        return rg.lora_check_device_errors(self.pool.handle, check=False)


def close(got, want, tol, dt, what):
    got = got.detach().to("cpu", torch.float64).numpy()
    rows = ~np.isnan(want)
    bad = np.abs(got - want) > tol * (1 + kv_ref.HALF[dt]) + kv_ref.HALF[dt] * np.abs(want) + 1e-30
    bad &= rows
    assert np.isfinite(got[rows]).all(), what
    worst = np.max(np.where(rows, np.abs(got - want) / (tol + kv_ref.HALF[dt] * np.abs(want) + 1e-30), 0)) if rows.any() else 0
    say(f"{what}: worst error {worst:.3f} of the bound")
    assert not bad.any(), (what, int(bad.sum()), worst)


def check(c, scores=True):
    want, tol, sw, stol = c.ref()
    canary = torch.full((c.T, c.width), 7.25, dtype=c.dt, device="cuda")
    prior = torch.rand((c.n, c.cap), generator=c.g, device="cuda") if scores else None
    sc = torch.full((c.n, c.cap), -3.0, device="cuda") if scores else None
    out = c.run(scores=sc, prior=prior, out=canary)
    torch.cuda.synchronize()
    assert c.errors() == 0, rg.lora_last_error()
    close(out, want, tol, c.dt, "out")
    outside = np.isnan(want).all(1)
    assert (canary.cpu()[torch.as_tensor(outside)] == 7.25).all(), "a row outside every sequence changed"
    if scores:
        held = np.arange(c.cap)[None] < np.asarray(c.lens)[:, None]
        assert (sc.cpu().numpy()[~held] == -3.0).all(), "scores behind a sequence's last token changed"
        p = prior.cpu().numpy().astype(np.float64)
        no_rows = np.zeros(c.n, bool) if c.q_start is None else np.diff(c.q_start) == 0
        w = np.where(held, p + sw, np.nan)
        close(sc, w, stol + kv_ref.EPS32 * np.abs(p + sw), torch.float32, f"scores ({no_rows.sum()} without rows)")
        again = prior.clone()                                  # in place, bit for bit the same
        out2 = c.run(scores=again, prior=again)
        assert torch.equal(again[torch.as_tensor(held)], sc[torch.as_tensor(held)])
        got = torch.as_tensor(~outside)
        assert torch.equal(out2[got].view(torch.uint8), out[got].view(torch.uint8))
    return out


LENS = [1, 0, 2, 31, 32, 33, 63, 64, 65, 127, 129, 200, 255, 257]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", list(GEO))
def test_attend_lengths(geo, dtype):
    check(Case(geo, dtype, LENS))


@pytest.mark.parametrize("dtype,geo,lens", [
    ("bf16", "gqa64", [1]), ("bf16", "mha128", [1]), ("f32", "mha64", [1]), ("bf16", "mqa128", [0]), ("bf16", "mha64", [0, 0, 5]),
    ("bf16", "gqa64", [3000]), ("f32", "gqa64", [2777]), ("bf16", "mqa128", [4099, 3]), ("bf16", "group20", [2049]),
    ("bf16", "dim256", [1025, 1, 0, 700]), ("bf16", "mha64", [5, 1900, 0, 0, 64, 513] * 7), ("bf16", "group16", [33] * 300),
])
def test_attend_shapes(geo, dtype, lens):
    check(Case(geo, dtype, lens, seed=3))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", list(GEO))
def test_chunk_lengths(geo, dtype):
    new = [1, 0, 2, 31, 1, 33, 40, 64, 65, 100, 3, 200, 17, 130]
    check(Case(geo, dtype, LENS, new, gap=2))


@pytest.mark.parametrize("dtype,geo,lens,new", [
    ("bf16", "mha64", [1], [1]), ("bf16", "mha128", [300], [300]), ("bf16", "gqa64", [1500], [3]), ("f32", "gqa64", [900], [260]),
    ("bf16", "mqa128", [700, 0, 9], [513, 0, 9]), ("bf16", "dim256", [600], [257]), ("bf16", "group20", [300, 300], [150, 300]),
    ("bf16", "group16", [129] * 40, [5] * 40), ("bf16", "group3", [1030], [1030]), ("bf16", "mha64", [0, 0, 4], [0, 3, 4]),
    ("bf16", "mha64", [2100, 40], [64, 40]),
])
def test_chunk_shapes(geo, dtype, lens, new):
    check(Case(geo, dtype, lens, new, seed=4, gap=1))


@pytest.mark.parametrize("geo,lens,new", [
    ("wide64", [300, 1, 0, 257, 128], [300, 1, 0, 129, 128]), ("wide64", [613, 5], [513, 5]),       # longer than the addresses kept
    ("wide64_kv64", [200, 97, 290], [200, 33, 290]), ("wide64_kv128", [401, 129], [384, 129]),
    ("wide128", [260, 384, 385], [260, 384, 385]), ("wide128_kv32", [390, 0, 7, 400, 300], [390, 0, 7, 400, 300]),
    ("wide64", [513], [513]), ("wide64", [64] * 9, [64] * 9),
])
def test_chunk_pairs(geo, lens, new):
    """Query tiles taken two a workgroup: odd and even numbers of them, sequences of one, none, and long ones."""
    c = Case(geo, "bf16", lens, new, seed=6, gap=1)
    group = c.layout.n_heads // c.layout.n_kv_heads
    hpw = 4 if group % 4 == 0 else 2 if group % 2 == 0 else 1
    assert c.layout.n_heads // hpw * (c.T // (128 // hpw)) >= 1024
    check(c)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo,lens,new", [
    ("gqa64", [5000, 0, 257, 1, 256, 2], [1, 0, 3, 1, 0, 2]), ("mqa128", [2500], [40]), ("group20", [1300, 511], [33, 1]),
    ("dim256", [1025, 300], [7, 129]), ("group3", [900, 0, 513], [130, 2, 257]), ("mha64", [777] * 5, [3] * 5),
])
def test_chunk_ranges(geo, lens, new, dtype):
    """Few rows on long caches: the tokens are cut into ranges, joined afterwards."""
    if 0 in lens and new[lens.index(0)]:                        # a padded row that has new tokens: recorded, zero rows
        c = Case(geo, dtype, lens, new, seed=8, gap=1)
        want, tol, _, _ = c.ref()
        out = c.run(out=torch.full((c.T, c.width), 7.25, dtype=c.dt, device="cuda"))
        close(out, want, tol, c.dt, "out")
        return
    check(Case(geo, dtype, lens, new, seed=8, gap=1))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("at", [0, 255, 256, 700, 990, 999])
def test_chunk_ranges_pass_infinities(at, dtype):
    """An infinite value reaches the rows from its own on, whichever range holds it, and no other."""
    c = Case("gqa64", dtype, [1000], [20])
    want, tol, _, _ = c.ref()
    tpp, dim = c.layout.tokens_per_page, c.layout.head_dim
    c.pool.pages[int(c.table[0, 1, at // tpp]), (at % tpp) * 2 * dim + 3] = float("inf")
    out = c.run().cpu().to(torch.float64).numpy()
    hit = np.zeros(want.shape, bool)
    for h in range(4):
        hit[max(0, at - 980):, h * dim + 3] = True
    assert (out[hit] == np.inf).all()
    want[hit] = out[hit] = 0
    close(torch.as_tensor(out), want, tol, c.dt, "out")


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [40, 130, 300])
def test_chunk_pairs_hide_what_comes_later(at, value):
    """A value that is not finite reaches the rows from its own position on, in either tile of a pair, and no other."""
    c = Case("wide64", "bf16", [384, 140], [384, 140], seed=7)
    want, tol, _, _ = c.ref()
    c.pool.pages[int(c.table[0, 1, at]), 64 * 9 + 3] = value
    out = c.run()
    hit = np.zeros(want.shape, bool)
    hit[at:384, 64 * 9 + 3] = True
    got = out.cpu().to(torch.float64).numpy()
    assert (np.isnan(got[hit]) if value != value else got[hit] == value).all()
    want[hit] = 0
    close(torch.as_tensor(np.where(hit, 0, got)), want, np.where(hit, 1, tol), c.dt, "out")


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("new", [None, [50, 97, 1, 64]])
def test_any_scale(new, scale):
    """A scale of zero weighs all tokens alike; a negative one turns the order round."""
    c = Case("gqa64", "bf16", [50, 129, 300, 64], new)
    c.scale = scale
    want, tol, sw, stol = c.ref()
    sc = torch.zeros((c.n, c.cap), device="cuda")
    close(c.run(scale=scale, scores=sc), want, tol, c.dt, "out")
    close(sc, sw, stol, torch.float32, "scores")


@pytest.mark.parametrize("new", [None, [50, 129, 1, 64]])
def test_rows_of_a_wider_matrix(new):
    """q and out as column ranges of wider buffers: the columns beside them stay as they were."""
    c = Case("gqa64", "bf16", [50, 129, 300, 64], new)
    wide = torch.full((c.T, 3 * c.width), 5.0, dtype=c.dt, device="cuda")
    wide[:, c.width:2 * c.width] = c.q
    res = torch.full((c.T, 2 * c.width), 9.0, dtype=c.dt, device="cuda")
    out = c.run(q=wide[:, c.width:2 * c.width], out=res[:, :c.width])
    want, tol, _, _ = c.ref()
    close(out, want, tol, c.dt, "strided")
    assert (res[:, c.width:] == 9.0).all()


@pytest.mark.parametrize("geo", ["mha64", "mqa128"])
@pytest.mark.parametrize("new", [None, [3, 40]])
def test_values_behind_the_last_token_are_not_read(geo, new):
    """NaN and infinities in page space that no token of the sequence owns change nothing."""
    c = Case(geo, "bf16", [37, 66], new)
    tpp, w = c.layout.tokens_per_page, c.layout.n_kv_heads * c.layout.head_dim
    clean = c.run()
    used = torch.zeros(c.pool.pages.shape, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lens):
        for t in range(n):
            for r in range(2):
                used[int(c.table[b, r, t // tpp]), (t % tpp) * w:(t % tpp + 1) * w] = True
    c.pool.pages[~used] = float("nan")
    assert torch.equal(c.run(), clean)
    c.pool.pages[~used] = float("inf")
    assert torch.equal(c.run(), clean)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_bad_token_reaches_no_row_before_it(which, value, dtype):
    c = Case("gqa64", dtype, [150], [150])
    want, tol, _, _ = c.ref()
    at = 70
    tpp, w, dim = c.layout.tokens_per_page, c.layout.n_kv_heads * c.layout.head_dim, c.layout.head_dim
    page = int(c.table[0, 0 if which == "k" else 1, at // tpp])
    c.pool.pages[page, (at % tpp) * w + dim + 3] = value       # second K/V head, element 3
    sc = torch.zeros((1, c.cap), device="cuda")
    out = c.run(scores=sc)
    want[at:] = np.nan                                          # rows from `at` on are checked below
    close(out, want, tol, c.dt, "rows before")
    heads, group = c.layout.n_heads, c.layout.n_heads // c.layout.n_kv_heads
    rows = out[at:].float().view(-1, heads, dim)
    assert torch.isfinite(rows[:, :group]).all()                # the first K/V head's rows are clean
    if which == "v":
        x = rows[:, group:, 3]
        assert (torch.isnan(x) if value != value else x == value).all()
        assert torch.isfinite(rows[:, group:, :3]).all() and torch.isfinite(rows[:, group:, 4:]).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("at", [0, 5, 31, 40, 63, 64])
def test_an_infinite_value_stays_infinite(at, dtype):
    """In the rows from its own on, also where it lies in the first tokens that a row weighs."""
    c = Case("gqa64", dtype, [150], [150])
    want, tol, _, _ = c.ref()
    tpp, dim = c.layout.tokens_per_page, c.layout.head_dim
    c.pool.pages[int(c.table[0, 1, at // tpp]), (at % tpp) * 2 * dim + 3] = float("inf")   # first K/V head, element 3
    out = c.run().cpu().to(torch.float64).numpy()
    hit = np.zeros(want.shape, bool)
    for h in range(4):
        hit[at:, h * dim + 3] = True
    assert (out[hit] == np.inf).all()
    want[hit] = out[hit] = 0
    close(torch.as_tensor(out), want, tol, c.dt, "out")


def test_attend_values_pass_through():
    """Infinities and NaN of a token that is seen come through as the formula has them."""
    c = Case("mha64", "bf16", [90, 90, 90, 64])
    d = 64
    c.pool.pages[int(c.table[0, 1, 40]), 5] = float("inf")      # a value
    c.pool.pages[int(c.table[1, 1, 41]), 6] = float("nan")
    c.pool.pages[int(c.table[2, 0, 42]), 7] = float("nan")      # a key: the whole head of that sequence
    c.pool.pages[torch.as_tensor(c.table[3, 0, :64].astype(np.int64), device="cuda"), 0:d] = float("-inf")
    c.q[3, :d] = 1.0                                            # head 0 of sequence 3: every product is -inf
    out = c.run().float()
    assert out[0, 5] == float("inf") and torch.isnan(out[1, 6])
    assert torch.isnan(out[2, :d]).all() and torch.isfinite(out[2, d:]).all()
    assert (out[3, :d] == 0).all() and torch.isfinite(out[3, d:]).all()
    ok = torch.ones_like(out, dtype=torch.bool)
    ok[0, 5] = ok[1, 6] = False
    ok[2, :d] = False
    assert torch.isfinite(out[ok]).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("new", [None, [4, 60, 64]])
def test_large_logits(new, dtype):
    """Logits of hundreds, one token far above the rest: the running maximum keeps every weight in range."""
    c = Case("mha64", dtype, [100, 60, 333], new)
    c.q.mul_(30.0)
    check(c)


@pytest.mark.parametrize("new", [None, [5, 70]])
def test_bad_pages_and_lengths_are_recorded(new):
    c = Case("gqa64", "bf16", [50, 70], new, extra_pages=4)
    c.table[0, 0, 3] = c.pool.num_pages
    c.table[1, 1, 5] = -1
    c.d_table = c.dev(c.table)
    sc = torch.zeros((2, c.cap), device="cuda")
    out = c.run(scores=sc)
    want, tol, sw, stol = c.ref()
    close(out, want, tol, c.dt, "bad pages are absent")
    assert (sc.cpu().numpy()[0, 6:8] == 0).all() and (sc.cpu().numpy()[1, 10:12] == 0).all()
    assert c.errors() == rg.LORA_EDEVICE and "page-id" in rg.lora_last_error()
    for lens in ([c.cap + 1, 70], [-1, 70]) + (([4, 70],) if new else ()):
        c.d_lens = c.dev(lens)
        out = c.run()
        rows = slice(0, 1) if new is None else slice(0, 5)
        assert (out[rows] == 0).all() and (out[rows.stop:] != 0).any()
        assert c.errors() == rg.LORA_EDEVICE and "length" in rg.lora_last_error()
    c.d_lens = c.dev([50, 70])
    if new is None:
        run = lambda: c.run(max_len=60)                         # a length above max_len
        out = run()
        assert (out[1] == 0).all() and (out[0] != 0).any() and c.errors() == rg.LORA_EDEVICE
    else:
        for starts in ([0, 5, 76], [0, 80, 75], [-2, 5, 75]):   # ranges that leave [0, T] or run backwards
            c.d_start = c.dev(starts)
            canary = torch.full((c.T, c.width), 7.25, dtype=c.dt, device="cuda")
            c.run(out=canary)
            assert c.errors() == rg.LORA_EDEVICE
            assert (canary == 7.25).any()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", ["mha64", "mqa128", "dim256", "mha128"])
@pytest.mark.parametrize("new", [None, [1, 0, 5, 33, 2]])
def test_write(geo, dtype, new):
    c = Case(geo, dtype, [9, 0, 5, 77, 64], new, gap=0 if new is None else 3)
    w, tpp = c.layout.n_kv_heads * c.layout.head_dim, c.layout.tokens_per_page
    kv = torch.empty((c.T, 3 * w), dtype=c.dt, device="cuda").normal_(generator=c.g)
    k, v = kv[:, :w], kv[:, 2 * w:]
    want = c.pool.pages.clone()
    starts = list(range(c.n + 1)) if new is None else c.q_start
    for b, n in enumerate(c.lens):
        m = starts[b + 1] - starts[b]
        for i in range(m if n else 0):
            t = n - m + i
            for r, rows in enumerate((k, v)):
                want[int(c.table[b, r, t // tpp]), (t % tpp) * w:(t % tpp + 1) * w] = rows[starts[b] + i]
    c.pool.kv_write(c.layout, k, v, c.d_table, c.d_lens, c.d_start)
    torch.cuda.synchronize()
    assert c.errors() == 0
    assert torch.equal(c.pool.pages.view(torch.uint8), want.view(torch.uint8))


def test_write_skips_bad_pages():
    c = Case("gqa64", "bf16", [5, 6])
    c.table[1, 1, 2] = -7
    c.d_table = c.dev(c.table)
    w = c.layout.n_kv_heads * c.layout.head_dim
    k = torch.ones((2, w), dtype=c.dt, device="cuda")
    want = c.pool.pages.clone()
    for r in range(2):
        want[int(c.table[0, r, 2]), :w] = 1
    c.pool.kv_write(c.layout, k, k, c.d_table, c.d_lens)
    assert torch.equal(c.pool.pages.view(torch.uint8), want.view(torch.uint8))
    assert c.errors() == rg.LORA_EDEVICE


def test_far_pages():
    """Pages behind the first 4 GiB of the pool."""
    layout = rg.lora_kv_layout_t(4, 4, 64, 1)
    H, P = 4096, 700_000
    pool = rg.Pool(P, H, rg.LORA_BF16, max_rank=1)
    n = 77
    ids = np.arange(P - 2 * n, P, dtype=np.int32).reshape(1, 2, n)
    pool.pages[P - 2 * n:].normal_()
    k = torch.randn((n, 256), device="cuda").bfloat16()
    v = torch.randn((n, 256), device="cuda").bfloat16()
    q = torch.randn((n, 256), device="cuda").bfloat16()
    t, lens, starts = (torch.as_tensor(np.asarray(x, np.int32), device="cuda") for x in (ids, [n], [0, n]))
    pool.kv_write(layout, k, v, t, lens, starts)
    assert torch.equal(pool.pages[P - 2 * n:P - n, :256], k) and torch.equal(pool.pages[P - n:, :256], v)
    out = pool.kv_attend_chunk(layout, q, t, lens, starts)
    want, tol, _, _ = kv_ref.attend(pool.pages, layout, q, ids, [n], [0, n], 0.125, 2.0 ** -8)
    close(out, want, tol, torch.bfloat16, "far chunk")
    out = pool.kv_attend(layout, q[-1:], t, lens)
    want, tol, _, _ = kv_ref.attend(pool.pages, layout, q[-1:], ids, [n], None, 0.125, 2.0 ** -15)
    close(out, want, tol, torch.bfloat16, "far token")
    assert rg.lora_check_device_errors(pool.handle, check=False) == 0


def _evict_case(tpp, layers, lens, seed, kind):
    rng = np.random.default_rng(seed)
    mp = max(1, max(-(-n // tpp) for n in lens)) + 2
    table = rng.permutation(layers * len(lens) * 2 * mp).astype(np.int32).reshape(layers, len(lens), 2, mp)
    scores = rng.random((layers, len(lens), mp * tpp)).astype(np.float32)
    if kind == "ties":
        scores = np.floor(scores * 4).astype(np.float32)
    elif kind == "special":
        pick = rng.integers(0, 6, scores.shape)
        scores = np.where(pick == 0, np.float32(np.nan), np.where(pick == 1, np.float32(-0.0), np.where(
            pick == 2, np.float32(0.0), np.where(pick == 3, np.float32(-1.5), scores)))).astype(np.float32)
    elif kind == "narrow":
        scores = (np.float32(1.0) + scores * np.float32(2.0 ** -20)).astype(np.float32)
    return table, scores


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["random", "ties", "special", "narrow"])
@pytest.mark.parametrize("tpp,layers,lens,budget,first,last,max_drop", [
    (1, 2, [0, 1, 5, 300, 64, 1025, 2500], 40, 4, 8, None),
    (1, 1, [4097], 1, 0, 0, None),
    (1, 3, [700, 30], 100, 0, 0, 57),
    (4, 2, [0, 3, 4, 5, 401, 1000], 33, 3, 10, None),
    (5, 1, [5003, 77], 70, 6, 1, 400),
    (256, 1, [3000], 300, 1, 1, None),
    (1, 1, [100, 200], 300, 4, 4, None),
    (2, 1, [100], 0, 60, 60, None),
    (1, 2, [511, 512, 3, 505], 100, 2, 2, None),
    (1, 1, [2040, 1999], 1000, 2, 2, None),
    (1, 1, [9001, 20], 4000, 4, 8, None),                   # rows that do not fit the registers of a workgroup
    (2, 1, [17003, 500], 301, 5, 9, 7000),
])
def test_evict(tpp, layers, lens, budget, first, last, max_drop, kind, in_place):
    pool = rg.Pool(4, 64 * 256, rg.LORA_BF16, max_rank=1)
    layout = rg.lora_kv_layout_t(1, 1, 64, tpp)
    table, scores = _evict_case(tpp, layers, lens, 11, kind)
    mp = table.shape[-1]
    lens_in = list(lens) + [-1, mp * tpp + 1]                   # two rows out of range: left as they are
    table = np.concatenate([table, table[:, :2][:, [0, 0]] if table.shape[1] < 2 else table[:, :2]], 1)
    scores = np.concatenate([scores, scores[:, [0, 0]]], 1)
    want = kv_ref.evict(layout, table, scores, lens_in, budget, first, last, max_drop or mp)
    d_t, d_s, d_l = (torch.as_tensor(x, device="cuda") for x in (table.copy(), scores.copy(), np.asarray(lens_in, np.int32)))
    got = pool.kv_evict(layout, d_t, d_s, d_l, budget, first, last, max_drop, in_place=in_place)
    torch.cuda.synchronize()
    assert rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_EDEVICE
    if in_place:
        assert got[0] is d_t and got[1] is d_s
    else:
        assert np.array_equal(d_t.cpu().numpy(), table)
    for name, g, w in zip(("table", "scores", "lens", "dropped", "n_dropped"), got, want):
        g = g.cpu().numpy()
        same = (g.view(np.int32) == w.view(np.int32)) | ((g == 0) & (w == 0)) if name == "scores" else g == w
        assert same.all(), (name, np.argwhere(~same)[:5].tolist())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", ["mha64", "mqa128"])
def test_a_run_of_them_together(geo, dtype):
    """Prompts, decode steps, eviction, more steps, a request that finishes and one that takes its place: the
    cache against a float64 model that keeps the kept tokens' K and V itself."""
    nh, nkv, dim, H, tpp = GEO[geo]
    layers, rows = 2, 3
    layout = rg.lora_kv_layout_t(nh, nkv, dim, tpp)
    pool = rg.Pool(2 * layers * 3 * (140 // tpp + 3), H, rg.LORA_BF16 if dtype == "bf16" else rg.LORA_F32, max_rank=1)
    cache = rg.KvCache(pool, layers, layout, rows, 140, scores=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    K = {}                                     # (request, layer) -> list of (k, v) rows, score array

    def step(counts):
        cache.append(counts)
        chunk = max(counts.values()) > 1
        by_row = sorted(counts, key=lambda r: cache.rows[r])
        T = sum(counts.values()) if chunk else rows
        for layer in range(layers):
            k, v, q = (torch.empty((T, n * dim), dtype=DT[dtype], device="cuda").normal_(generator=g)
                       for n in (nkv, nkv, nh))
            cache.write(layer, k, v)
            out = cache.attend(layer, q)
            at = 0
            for rid in by_row:
                m = counts[rid]
                sl = slice(at, at + m) if chunk else slice(cache.rows[rid], cache.rows[rid] + 1)
                at += m
                held = K.setdefault((rid, layer), [torch.empty((0, nkv * dim), dtype=DT[dtype], device="cuda")] * 2 + [np.zeros(0)])
                held[0], held[1] = torch.cat([held[0], k[sl]]), torch.cat([held[1], v[sl]])
                n = held[0].shape[0]
                one = rg.lora_kv_layout_t(nh, nkv, dim, 1)
                want, tol, sw, stol = kv_ref.attend(torch.cat([held[0], held[1]]), one, q[sl],
                                                    np.arange(2 * n, dtype=np.int32).reshape(1, 2, n), [n], [0, m], dim ** -0.5,
                                                    kv_ref.ROUNDED[DT[dtype], chunk])
                close(out[sl], want, tol, DT[dtype], f"request {rid} layer {layer} ({n} tokens)")
                held[2] = np.concatenate([held[2], np.zeros(m)]) + sw[0]
            if not chunk:
                idle = [r for r in range(rows) if r not in [cache.rows[x] for x in counts]]
                assert (out[idle] == 0).all()

    def check_scores():
        for (rid, layer), (_, _, s) in K.items():
            got = cache.scores[layer, cache.rows[rid]].cpu().numpy().astype(np.float64)
            assert np.allclose(got[: s.size], s, rtol=1e-3, atol=1e-4) and (got[s.size:] == 0).all()

    def evict(budget, first, last):
        before = rg.lora_pool_stats(pool.handle)["free_pages"]
        old = cache.scores.cpu().numpy().copy()
        gone = cache.evict(budget, first, last)
        for (rid, layer), held in K.items():
            n = held[0].shape[0]
            s = old[layer, cache.rows[rid]][None, None, :]
            mp = s.size // tpp
            t = np.arange(2 * mp, dtype=np.int32).reshape(1, 1, 2, mp)
            kept = kv_ref.evict(layout, t, s, [n], budget, first, last, mp)[0][0, 0, 0]
            toks = [p * tpp + j for p in kept if p >= 0 for j in range(tpp) if p * tpp + j < n]
            assert n - len(toks) == gone.get(rid, 0)
            pick = torch.as_tensor(toks, device="cuda")
            held[0], held[1], held[2] = held[0][pick], held[1][pick], held[2][toks]
        pages = sum(2 * layers * (n // tpp) for n in gone.values())
        assert rg.lora_pool_stats(pool.handle)["free_pages"] == before + pages
        for rid, row in cache.rows.items():
            ids = sorted(int(x) for x in cache.table[:, row].cpu().numpy().reshape(-1) if x >= 0)
            assert ids == sorted(rg.lora_pool_kv_pages(pool.handle, rid))
        return gone

    step({7: 60, 9: 33})
    for _ in range(3):
        step({7: 1, 9: 1})
    check_scores()
    assert evict(40, 2, 5)
    check_scores()
    step({7: 1})
    step({7: 1, 9: 1, 4: 1})
    step({4: 50, 9: 2})
    check_scores()
    cache.finish(9)
    for key in [k for k in K if k[0] == 9]:
        del K[key]
    step({11: 45})
    step({11: 1, 7: 1, 4: 1})
    assert evict(30, 1, 1)
    check_scores()
    step({11: 1, 7: 1, 4: 1})
    for rid in (4, 7, 11):
        cache.finish(rid)
    st = rg.lora_pool_stats(pool.handle)
    assert st["kv_pages"] == 0 and st["free_pages"] == pool.num_pages
    assert (cache.table == -1).all() and (cache.scores == 0).all()
    assert rg.lora_check_device_errors(pool.handle, check=False) == 0


def test_append_short_of_pages_changes_nothing():
    layout = rg.lora_kv_layout_t(4, 4, 64, 1)
    pool = rg.Pool(2 * 2 * 10, 256, rg.LORA_BF16, max_rank=1)
    cache = rg.KvCache(pool, 2, layout, 2, 20)
    cache.append({1: 6})
    free, table = rg.lora_pool_free_list(pool.handle), cache.table.clone()
    with pytest.raises(rg.LoraError) as e:
        cache.append({1: 2, 2: 9})
    assert e.value.status == "enomem"
    assert sorted(rg.lora_pool_free_list(pool.handle)) == sorted(free) and torch.equal(cache.table, table)
    assert cache.rows == {1: 0} and cache.length == [6, 0] and cache.lens.tolist() == [6, 0]
    for bad in ({1: 0}, {1: 15}, {2: 1, 3: 1}):
        with pytest.raises(ValueError):
            cache.append(bad)
    cache.append({1: 2, 2: 2})
    assert cache.lens.tolist() == [8, 2]


@pytest.mark.parametrize("new", [None, [20, 33, 64, 1]])
def test_captured_and_replayed(new):
    """Two captured calls with other work between the replays: lengths, pages and queries change, the graphs
    read them at replay; each replay equals the eager call, bit for bit."""
    c = Case("gqa64", "bf16", [40, 33, 500, 64], new, extra_pages=0)
    d = Case("mha64", "bf16", [90, 33, 200, 64], new, seed=9)
    outs, graphs = [], []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sc = [torch.zeros((x.n, x.cap), device="cuda") for x in (c, d)]
    with torch.cuda.stream(s):
        for x, z in zip((c, d), sc):
            x.run(scores=z)
            x.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for x, z in zip((c, d), sc):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.run(scores=z))
        graphs.append(g)
    for turn in range(4):
        for x in (c, d):
            x.q.copy_(torch.randn_like(x.q.float()).to(x.dt))
            new_lens = [max(n - 3 * turn, 0 if new is None else n - (0 if m + 3 * turn > n else 3 * turn)) for n, m in
                        zip(x.lens, new or [1] * x.n)]
            x.d_lens.copy_(x.dev(new_lens))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        scores = [z.clone() for z in sc]
        for x, z, o, w in zip((c, d), sc, got, scores):
            eager = torch.zeros_like(z)
            assert torch.equal(x.run(scores=eager), o), turn
            held = torch.arange(x.cap, device="cuda")[None] < x.d_lens[:, None]
            assert torch.equal(eager[held], w[held])
        assert c.errors() == 0 and d.errors() == 0


@pytest.mark.parametrize("geo,lens,new", [("gqa64", [2600, 900, 40], [20, 65, 3]), ("wide64", [300, 257], [300, 257])])
def test_captured_chunks_of_other_lengths(geo, lens, new):
    """Ranges and pairs: how the rows are shared out and how long the caches are is read at the replay."""
    c = Case(geo, "bf16", lens, new, seed=11, extra_pages=0)
    sc = torch.zeros((c.n, c.cap), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(scores=sc)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.run(scores=sc)
    for turn in range(4):
        m = [new[0] - 3 * turn] + [new[1] + 2 * turn if lens[1] > new[1] + 6 else new[1]] + new[2:]
        c.d_start.copy_(c.dev(np.cumsum([0] + m)))
        c.d_lens.copy_(c.dev([max(x, n - 200 * turn) if turn < 3 else (0 if b == 1 else n) for b, (n, x) in enumerate(zip(lens, m))]))
        c.q.copy_(torch.randn_like(c.q.float()).to(c.dt))
        out.fill_(7.25)
        sc.zero_()
        g.replay()
        torch.cuda.synchronize()
        eager_out, eager = torch.full_like(out, 7.25), torch.zeros_like(sc)
        c.run(scores=eager, out=eager_out)
        assert torch.equal(out, eager_out) and torch.equal(sc, eager), turn
        c.errors()                                              # (the turn with an unused row that has new tokens)


def test_streams_of_their_own():
    """Calls on two streams at once, given as stream objects and as a handle, share no workspace."""
    c = Case("gqa64", "bf16", [700, 33, 1500])
    want = c.run()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(20):
        for s in (a, b.cuda_stream):
            sc = torch.zeros((c.n, c.cap), device="cuda")
            torch.cuda.synchronize()
            outs.append(c.run(scores=sc, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_python_refusals():
    c = Case("gqa64", "bf16", [5, 6])
    for kw in (dict(q=c.q.float()), dict(q=c.q[:, :-1]), dict(q=c.q[:1]), dict(scores=torch.zeros((2, 3), device="cuda")),
               dict(out=torch.empty((2, c.width), device="cuda")), dict(q=c.q.cpu())):
        with pytest.raises(ValueError):
            c.run(**kw)
    for kw in (dict(max_len=0), dict(max_len=c.cap + 1), dict(scale=float("inf")), dict(out=c.q),
               dict(prior=torch.zeros((2, c.cap), device="cuda"))):
        with pytest.raises(rg.LoraError) as e:
            c.run(**kw)
        assert e.value.code == rg.LORA_EINVAL
    assert c.errors() == 0
