"""The KV-cache attention calls in every form that a rule on sizes can choose, and several of them at once, on the
device, against plain float64 forms (kv_ref.py)."""
import numpy as np
import pytest
import torch

import rank_gemm_unified_amd as rg
from test_gpu_kv import DT, GEO, LENS, WIDE, Case, _gpu, check  # noqa: F401

pytestmark = pytest.mark.gpu

# 16 query heads on one K/V head of 256: the most LDS that the one-launch form takes at that head dim
WIDE["group16_256"] = (16, 1, 256, 256, 1)
ALL = [*GEO, "group16_256"]


def one_launch(c, max_len=None):
    """Whether attention of one token without scores is one launch: few workgroups, a few tiles to a wave of each."""
    lay = c.layout
    group = lay.n_heads // lay.n_kv_heads
    workgroups = c.n * lay.n_kv_heads * -(-group // 16)
    tile = 16 if c.dt is torch.float32 and lay.head_dim > 64 else 32
    waves = 4 if lay.head_dim == 256 else 8
    return workgroups <= 256 and -(-(max_len or c.cap) // tile) <= (3 if workgroups < 64 else 4) * waves


def ranges(c):
    """Ranges that the tokens of a chunk are cut into, at most."""
    lay = c.layout
    group = lay.n_heads // lay.n_kv_heads
    hpw = 4 if group % 4 == 0 else 2 if group % 2 == 0 else 1
    rows = 128 // hpw
    tiles = (c.T + min(c.n, c.T) * (rows - 1)) // rows
    return max(1, min((256 if lay.head_dim == 256 else 512) // (lay.n_heads // hpw * tiles), c.cap // 256, 512))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", ALL)
def test_attend_without_scores_in_one_launch(geo, dtype):
    lens = [1, 0, 2, 31, 32, 33, 64, 129] + ([] if geo == "mha128" else [63, 65, 127, 150])
    c = Case(geo, dtype, lens, seed=41)
    assert one_launch(c)
    check(c, scores=False)


@pytest.mark.parametrize("dtype,geo,lens", [
    ("bf16", "mha64", [1000, 17, 0, 999] * 4), ("f32", "mha64", [1000, 17, 0, 999] * 4), ("bf16", "mqa128", [700, 3]),
    ("f32", "group16", [300]), ("bf16", "group16", [700, 1]), ("bf16", "group20", [7, 690]), ("f32", "dim256", [150, 77]),
    ("bf16", "dim256", [350, 129]), ("f32", "group3", [128] * 60), ("bf16", "group16_256", [333]), ("f32", "mha64", [1]),
    ("bf16", "gqa64", [0]), ("f32", "mqa128", [0, 0]), ("f32", "mha128", [203]), ("bf16", "mha128", [203]),
])
def test_attend_without_scores_in_one_launch_shapes(geo, dtype, lens):
    """The longest caches that the rule lets through, single and empty ones."""
    c = Case(geo, dtype, lens, seed=42)
    assert one_launch(c)
    check(c, scores=False)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo", ALL)
def test_attend_without_scores_in_ranges(geo, dtype):
    """Whole sequences in one range, and pieces of one sequence in several."""
    for lens in (LENS + [1300], [3000, 1, 0, 700]):
        c = Case(geo, dtype, lens, seed=43)
        assert not one_launch(c)
        check(c, scores=False)


@pytest.mark.parametrize("dtype,geo,lens", [
    ("f32", "mha64", [33] * 300), ("f32", "group16", [257] * 290), ("bf16", "dim256", [64, 0, 9] * 100), ("f32", "dim256", [40] * 140),
    ("f32", "mqa128", [4099, 3]), ("bf16", "group16", [2600]), ("f32", "group20", [2049]), ("bf16", "group3", [1, 1900, 0, 513] * 9),
])
def test_attend_without_scores_in_ranges_shapes(geo, dtype, lens):
    c = Case(geo, dtype, lens, seed=44)
    assert not one_launch(c)
    check(c, scores=False)


@pytest.mark.parametrize("dtype", list(DT))
def test_one_workspace_for_every_batch(dtype):
    """Made for the largest batch, it serves the smaller ones, one launch or two."""
    geo, most, longest = "gqa64", 32, 1020
    forms = set()
    ws = None
    for n in (most, 4, 1, 31, 16):
        c = Case(geo, dtype, [longest] * n, seed=45, extra_pages=2)
        if ws is None:
            size = rg.lora_kv_attend_workspace_size(c.pool.handle, c.layout, most, c.cap)
            assert size > 0
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        forms.add(one_launch(c))
        want = c.run()
        assert torch.equal(c.run(workspace=ws), want)
        assert c.errors() == 0
    assert forms == {False, True}


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo,lens,new,least", [
    ("gqa64", [40000], [1], 65), ("gqa64", [20000, 40000], [2, 1], 65), ("mqa128", [33000, 5], [3, 1], 65), ("dim256", [20000], [5], 65),
    ("mqa128", [131071], [2], 512),
])
def test_chunk_in_many_ranges(geo, lens, new, least, dtype):
    """More ranges than the join has lanes, and as many as there can be."""
    c = Case(geo, dtype, lens, new, seed=46, gap=1)
    assert ranges(c) >= least
    check(c)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("geo,lens,new", [("gqa64", [5000, 0, 257], [1, 3, 3]), ("mqa128", [0, 2500], [40, 40]), ("dim256", [1025, 0], [7, 9])])
def test_chunk_in_ranges_of_rows_without_a_cache(geo, lens, new, dtype):
    """New tokens of an unused row: zero rows."""
    c = Case(geo, dtype, lens, new, seed=47, gap=1)
    assert ranges(c) > 1
    check(c)


def _together(cases, calls):
    """calls: one per case and turn, on a stream per case, none waited for; every stream is busy at first, so that the
    calls behind run at the same time."""
    want = []
    for c in cases:
        sc = torch.zeros((c.n, c.cap), device="cuda")
        want.append((c.run(scores=sc).clone(), sc, c.run().clone()))
    streams = [torch.cuda.Stream() for _ in cases]
    busy = torch.randn((4096, 4096), device="cuda").bfloat16()
    got = [[] for _ in cases]
    sums = [[torch.zeros_like(w[1]) for _ in range(calls)] for w in want]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(8):
                torch.mm(busy, busy)
    for i in range(calls):
        for c, s, g, z in zip(cases, streams, got, sums):
            on = s if i % 2 else s.cuda_stream
            g.append((c.run(scores=z[i], stream=on), c.run(stream=on)))
    torch.cuda.synchronize()
    for c, w, g, z in zip(cases, want, got, sums):
        for i in range(calls):
            assert torch.equal(g[i][0], w[0]) and torch.equal(g[i][1], w[2]) and torch.equal(z[i], w[1]), (i, c.lens)
        assert c.errors() == 0


@pytest.mark.parametrize("dtype", list(DT))
def test_calls_at_the_same_time(dtype):
    """On streams of their own, tokens and chunks, whole, in ranges and in one launch: workspaces and scores do not mix."""
    _together([Case("gqa64", dtype, [700, 33, 1500], seed=51), Case("gqa64", dtype, [1500, 700, 33], seed=52),
               Case("gqa64", dtype, [900, 300], [20, 9], seed=53), Case("gqa64", dtype, [300, 900], [9, 20], seed=54)], 12)


def test_calls_of_one_pool_at_the_same_time():
    """One pool and one table, other queries."""
    a = Case("mqa128", "bf16", [700, 33, 1500], seed=55)
    b = Case("mqa128", "bf16", [700, 33, 1500], seed=55)
    b.pool, b.d_table, b.table = a.pool, a.d_table, a.table
    b.q.normal_(generator=b.g)
    _together([a, b], 20)


@pytest.mark.parametrize("new", [None, [20, 9]])
def test_graphs_replayed_at_the_same_time(new):
    """Two captured calls share no workspace: replayed on two streams at once, several times."""
    cases = [Case("gqa64", "bf16", lens, new, seed=seed, extra_pages=0) for lens, seed in (([900, 1300], 56), ([1300, 900], 57))]
    sums = [torch.zeros((c.n, c.cap), device="cuda") for c in cases]
    eager = [torch.zeros_like(z) for z in sums]
    want = [c.run(scores=z) for c, z in zip(cases, eager)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, z in zip(cases, sums):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run(scores=z))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    busy = torch.randn((4096, 4096), device="cuda").bfloat16()
    for turn in range(5):
        for o, z in zip(outs, sums):
            o.fill_(7.25)
            z.zero_()
        torch.cuda.synchronize()
        for s in streams:
            with torch.cuda.stream(s):
                for _ in range(4):
                    torch.mm(busy, busy)
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, o, w, z, e in zip(cases, outs, want, sums, eager):
            assert torch.equal(o, w) and torch.equal(z, e), turn


@pytest.mark.parametrize("new", [None, [3, 5]])
def test_workspaces_refused(new):
    """Memory of the host or with gaps never reaches a kernel; too little of it is the call's own refusal."""
    c = Case("gqa64", "bf16", [700, 1500], new)
    size = 1 << 24
    for ws in (torch.zeros(size, dtype=torch.uint8), torch.zeros(2 * size, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            c.run(workspace=ws)
    with pytest.raises(rg.LoraError):
        c.run(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert torch.equal(c.run(workspace=torch.zeros(size, dtype=torch.uint8, device="cuda")), c.run())
    assert c.errors() == 0
