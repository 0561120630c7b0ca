"""The KV-cache calls' host side on the CPU: refusals (every argument is checked before any device work, so
a bookkeeping-only pool and made-up addresses serve) and giving KV pages back to the pool."""
import ctypes

import numpy as np
import pytest

import rank_gemm_unified_amd as rg

A = 1 << 40            # an address that is never read: every call here is refused, or has nothing to do
GAP = 1 << 30


def _pool(hidden=256, pages=64):
    return rg.Pool(pages, hidden, rg.LORA_BF16, max_rank=1, device=None)


L = rg.lora_kv_layout_t(8, 2, 64, 2)
WRITE = dict(k=A, ldk=128, v=A + GAP, ldv=128, table=A + 2 * GAP, max_pages=4, q_start=A + 3 * GAP, lens=A + 4 * GAP, n_seq=3, T=5)
TOKEN = dict(q=A, ldq=512, table=A + GAP, max_pages=4, lens=A + 2 * GAP, n_seq=3, max_len=8, scale=0.125,
             out=A + 3 * GAP, ldo=512, prior=None, scores=A + 5 * GAP, workspace=A + 6 * GAP, workspace_bytes=1 << 29)
CHUNK = dict(TOKEN, q_start=A + 7 * GAP, T=5)
EVICT = dict(layers=2, n_seq=3, table=A, table_out=A, max_pages=4, scores=A + GAP, scores_out=A + GAP, lens=A + 2 * GAP,
             lens_out=A + 3 * GAP, budget=4, keep_first=1, keep_last=2, dropped=A + 4 * GAP, max_drop=4,
             n_dropped=A + 5 * GAP)
CALLS = {"write": (rg.lora_kv_write, WRITE), "token": (rg.lora_kv_attend, TOKEN), "chunk": (rg.lora_kv_attend_chunk, CHUNK),
         "evict": (rg.lora_kv_evict, EVICT)}


POOL = _pool()         # freeing a pool clears the last error: this one lives on


def _call(which, layout=L, **change):
    fn, args = CALLS[which]
    return fn(POOL.handle, layout, **dict(args, **change), stream=0, check=False)


@pytest.mark.parametrize("which", list(CALLS))
def test_good_arguments_reach_the_last_check(which):
    assert _call(which) == rg.LORA_EINVAL and "bookkeeping-only" in rg.lora_last_error()


@pytest.mark.parametrize("which", list(CALLS))
@pytest.mark.parametrize("layout", [
    (0, 1, 64, 1), (8, 3, 64, 1), (8, 0, 64, 1), (-8, -2, 64, 1), (8, 2, 96, 1), (8, 2, 0, 1), (8, 2, 64, 0), (8, 2, 64, 3), (8, 2, 256, 1),
    (8, 2, 64, 1 << 30), (1025, 1, 64, 1), (2, 2, 64, 257)])
def test_layouts_refused(which, layout):
    assert _call(which, layout=rg.lora_kv_layout_t(*layout)) == rg.LORA_EINVAL and "layout" in rg.lora_last_error()


REFUSED = [
    ("write", dict(k=None)), ("write", dict(v=None)), ("write", dict(table=None)), ("write", dict(lens=None)),
    ("write", dict(k=A + 8)), ("write", dict(ldk=127)), ("write", dict(ldk=132)), ("write", dict(ldv=-128)), ("write", dict(ldv=1 << 40)),
    ("write", dict(max_pages=0)), ("write", dict(max_pages=(1 << 21) + 1)), ("write", dict(n_seq=-1)),
    ("write", dict(n_seq=(1 << 16) + 1)), ("write", dict(T=-1)), ("write", dict(T=(1 << 22) + 1)),
    ("write", dict(q_start=None)), ("write", dict(q_start=A + 2)), ("write", dict(table=A + 2)), ("write", dict(lens=A + 1)),
    ("token", dict(q=None)), ("token", dict(out=None)), ("token", dict(table=None)), ("token", dict(lens=None)),
    ("token", dict(q=A + 2)), ("token", dict(ldq=511)), ("token", dict(ldq=516)), ("token", dict(ldo=448)), ("token", dict(out=A + 3 * GAP + 4)),
    ("token", dict(max_len=0)), ("token", dict(max_len=9)), ("token", dict(max_pages=-1)), ("token", dict(scale=float("nan"))),
    ("token", dict(scale=float("-inf"))), ("token", dict(out=A)), ("token", dict(out=A + 1024)), ("token", dict(prior=A + 5 * GAP + 4)),
    ("token", dict(prior=A + 8 * GAP, scores=None)), ("token", dict(scores=A + 5 * GAP + 1)),
    ("token", dict(workspace=None)), ("token", dict(workspace=A + 6 * GAP + 16)), ("token", dict(workspace_bytes=8)),
    ("chunk", dict(q_start=None)), ("chunk", dict(q_start=A + 1)), ("chunk", dict(T=(1 << 22) + 1)), ("chunk", dict(out=A + 2048)),
    ("chunk", dict(workspace_bytes=8)), ("chunk", dict(n_seq=-3)), ("chunk", dict(max_len=1 << 40)),
    ("token", dict(n_seq=65535, max_pages=1 << 21, max_len=1 << 20)), ("chunk", dict(n_seq=8192, max_pages=1 << 21, max_len=(1 << 21) + 1)),
    ("evict", dict(layers=0)), ("evict", dict(layers=65536)), ("evict", dict(n_seq=-1)), ("evict", dict(max_pages=0)), ("evict", dict(budget=-1)),
    ("evict", dict(keep_first=-1)), ("evict", dict(keep_last=-1)), ("evict", dict(max_drop=0)), ("evict", dict(max_drop=5)),
    ("evict", dict(keep_last=1 << 30)), ("evict", dict(lens_out=A + 2 * GAP)), ("evict", dict(table_out=A + 4)), ("evict", dict(scores_out=A + GAP + 32)),
    ("evict", dict(dropped=A)), ("evict", dict(n_dropped=A + 2 * GAP)), ("evict", dict(dropped=A + 5 * GAP - 4)),
] + [("evict", {k: None}) for k in ("table", "table_out", "scores", "scores_out", "lens", "lens_out", "dropped", "n_dropped")] \
  + [("evict", {k: A + 9 * GAP + 2}) for k in ("table", "scores_out", "lens_out", "n_dropped")]


@pytest.mark.parametrize("which,change", REFUSED, ids=[f"{w}-{'-'.join(map(str, c))}-{i}" for i, (w, c) in enumerate(REFUSED)])
def test_refused(which, change):
    assert _call(which, **change) == rg.LORA_EINVAL
    assert "bookkeeping-only" not in rg.lora_last_error() and "lora_kv" in rg.lora_last_error()


def test_null_pool_and_layout():
    for name, args in (("lora_kv_write", [None, ctypes.byref(L)]), ("lora_kv_write", [_pool().handle, None])):
        assert rg._lib.lora_kv_write(*args, A, 128, A, 128, A, 4, None, A, 1, 1, None) == rg.LORA_EINVAL
    assert rg.lora_kv_attend_workspace_size(None, L, 1, 1) == 0


def test_nothing_to_do_is_ok():
    for which, change in (("write", dict(T=0)), ("write", dict(n_seq=0, T=0, q_start=None)), ("token", dict(n_seq=0)),
                          ("chunk", dict(T=0)), ("chunk", dict(n_seq=0)), ("evict", dict(n_seq=0))):
        assert _call(which, **change) == 0


def test_workspace_sizes():
    p = _pool()
    for f in (lambda n, m, s: rg.lora_kv_attend_workspace_size(p.handle, L, n, m, s),
              lambda n, m, s: rg.lora_kv_attend_chunk_workspace_size(p.handle, L, 4, n, m, s)):
        assert f(0, 8, True) == 0 and f(1, 0, True) == 0 and f(1, (1 << 22) + 1, True) == 0 and f((1 << 22) + 1, 8, True) == 0
        assert 0 < f(1, 8, True) <= f(64, 8, True) <= f(64, 4096, True)
        assert f(64, 4096, False) <= f(64, 4096, True)
    assert rg.lora_kv_attend_workspace_size(p.handle, rg.lora_kv_layout_t(8, 3, 64, 1), 4, 8, True) == 0


def test_one_row_needs_no_stride():
    """A single row's distance to the next means nothing."""
    assert _call("write", T=1, n_seq=1, q_start=None, ldk=0, ldv=7) == rg.LORA_EINVAL
    assert "bookkeeping-only" in rg.lora_last_error()


def test_drop_kv_gives_pages_back():
    p = _pool(pages=40)
    a = [rg.lora_pool_grow_kv(p.handle, 5, 2) for _ in range(4)]
    b = rg.lora_pool_grow_kv(p.handle, 6, 2)
    free = rg.lora_pool_free_list(p.handle)
    go = [a[2][1], a[0][0], a[3][3]]
    assert rg.lora_pool_drop_kv(p.handle, 5, go) == 0
    held = [x for g in a for x in g]
    assert rg.lora_pool_kv_pages(p.handle, 5) == [x for x in held if x not in go]
    assert rg.lora_pool_free_list(p.handle) == free + go
    st = rg.lora_pool_stats(p.handle)
    assert st["kv_pages"] == 16 + 4 - 3 and st["free_pages"] == 40 - 17 and st["kv_requests"] == 2
    # the next pages handed out are the ones given back, latest first
    assert rg.lora_pool_grow_kv(p.handle, 6, 1) == go[::-1][:2]
    # refusals change nothing
    before = (rg.lora_pool_kv_pages(p.handle, 5), rg.lora_pool_free_list(p.handle), rg.lora_pool_stats(p.handle))
    for ids in ([b[0]], [a[1][0], a[1][0]], [a[1][0], go[0]], [-1], [a[1][0], 40]):
        assert rg.lora_pool_drop_kv(p.handle, 5, ids, check=False) == rg.LORA_EINVAL
    assert rg.lora_pool_drop_kv(p.handle, 99, [1], check=False) == rg.LORA_ENOENT
    assert rg._lib.lora_pool_drop_kv(p.handle, 5, None, 1) == rg.LORA_EINVAL
    assert rg._lib.lora_pool_drop_kv(p.handle, 5, None, -1) == rg.LORA_EINVAL
    assert rg._lib.lora_pool_drop_kv(None, 5, None, 0) == rg.LORA_EINVAL
    assert before == (rg.lora_pool_kv_pages(p.handle, 5), rg.lora_pool_free_list(p.handle), rg.lora_pool_stats(p.handle))
    assert rg.lora_pool_drop_kv(p.handle, 5, []) == 0
    # a request without pages stays known until it is freed
    assert rg.lora_pool_drop_kv(p.handle, 5, rg.lora_pool_kv_pages(p.handle, 5)) == 0
    assert rg.lora_pool_kv_pages(p.handle, 5) == []
    assert rg.lora_pool_free_kv(p.handle, 5) == 0 and rg.lora_pool_free_kv(p.handle, 6) == 0
    st = rg.lora_pool_stats(p.handle)
    assert st["kv_pages"] == 0 and st["free_pages"] == 40


def test_dropped_pages_serve_adapters():
    """One free list: what a cache gives back, an adapter can take."""
    p = rg.Pool(16, 64, rg.LORA_BF16, max_rank=4, device=None)
    for _ in range(8):
        rg.lora_pool_grow_kv(p.handle, 1, 1)
    assert rg.lora_pool_load_adapter(p.handle, 0, 2, None, None, 0, check=False) == rg.LORA_ENOMEM
    ids = rg.lora_pool_kv_pages(p.handle, 1)[2:6]
    assert rg.lora_pool_drop_kv(p.handle, 1, ids) == 0
    assert rg.lora_pool_load_adapter(p.handle, 0, 2, None, None, 0, check=False) == 0
    assert sorted(rg.lora_pool_adapter_pages(p.handle, 0)[0]) == sorted(ids)


def test_cache_needs_device_pages():
    import torch
    with pytest.raises(ValueError):
        rg.KvCache(_pool(), 2, L, 4, 100)
    z = torch.zeros((1, 2, 4), dtype=torch.int32)
    for call in (lambda: POOL.kv_write(L, z, z, z, z), lambda: POOL.kv_attend(L, z, z, z), lambda: POOL.kv_attend_chunk(L, z, z, z, z)):
        with pytest.raises(ValueError):
            call()


def test_reference_forms_agree_with_loops():
    """kv_ref against loops written out, on a small case."""
    import torch
    import kv_ref
    rng = np.random.default_rng(3)
    lay = rg.lora_kv_layout_t(4, 2, 64, 2)
    pages = torch.as_tensor(rng.standard_normal((20, 320)).astype(np.float32))
    table = rng.permutation(20).astype(np.int32).reshape(1, 2, 10)
    q = torch.as_tensor(rng.standard_normal((3, 256)).astype(np.float32))
    n = 7
    out, _, sc, _ = kv_ref.attend(pages, lay, q, table, [n], [0, 3], 0.3, 0.0)
    want_sc = np.zeros(n)
    for r in range(3):
        for h in range(4):
            k = [pages[int(table[0, 0, t // 2]), (t % 2) * 128 + h // 2 * 64:][:64].double().numpy() for t in range(n - 3 + r + 1)]
            v = [pages[int(table[0, 1, t // 2]), (t % 2) * 128 + h // 2 * 64:][:64].double().numpy() for t in range(n - 3 + r + 1)]
            x = np.array([0.3 * float(np.dot(q[r, h * 64:(h + 1) * 64].double().numpy(), kk)) for kk in k])
            p = np.exp(x - x.max())
            p /= p.sum()
            want_sc[: len(p)] += p
            assert np.allclose(out[r, h * 64:(h + 1) * 64], sum(a * b for a, b in zip(p, v)), atol=1e-12)
    assert np.allclose(sc[0, :n], want_sc, atol=1e-12) and (sc[0, n:] == 0).all()


def test_methods_refuse_a_bookkeeping_pool():
    import torch

    i32 = dict(dtype=torch.int32)
    table, lens, q = torch.zeros((3, 2, 4), **i32), torch.ones(3, **i32), torch.zeros((3, 512), dtype=torch.bfloat16)
    scores = torch.zeros((1, 3, 8))
    for call in (lambda: POOL.kv_write(L, q[:, :128], q[:, :128], table, lens),
                 lambda: POOL.kv_attend(L, q, table, lens),
                 lambda: POOL.kv_attend_chunk(L, q, table, lens, torch.arange(4, **i32)),
                 lambda: POOL.kv_evict(L, table[None], scores, lens, 4)):
        with pytest.raises(ValueError, match="bookkeeping-only"):
            call()


def test_chunk_workspace_of_the_largest_call_serves_all():
    size = lambda n, T, m, sc: rg.lora_kv_attend_chunk_workspace_size(POOL.handle, L, n, T, m, sc)
    for sc in (False, True):
        for m in (8, 255, 300, 512, 5000, 1 << 20):
            got = [size(4, T, m, sc) for T in (1, 3, 64, 500, 4096, 70000)]
            assert got == sorted(got)
        got = [size(4, 64, m, sc) for m in (8, 255, 300, 512, 5000, 1 << 20)]
        assert got == sorted(got)
        assert size(4, 64, 5000, sc) <= size(9, 64, 5000, sc)
