"""The calls of a step of drafted tokens, host side on the CPU: refusals (every argument is checked before any device
work, so a bookkeeping-only pool and made-up addresses serve), workspace sizes, and the plain forms' own checks."""
import ctypes
import itertools

import numpy as np
import pytest

import draft_ref
import rank_gemm_unified_amd as rg

A = 1 << 40            # an address that is never read: every call here is refused, or has nothing to do
GAP = 1 << 30
AT = [A + i * GAP for i in range(24)]

POOL = rg.Pool(64, 256, rg.LORA_BF16, max_rank=1, device=None)
L = rg.lora_kv_layout_t(8, 2, 64, 2)
ROPE = rg.lora_rope_t(AT[20], 100, 64, rg.LORA_ROPE_HALVES)
PLAN = dict(layers=2, n_seq=3, counts=AT[0], lens=AT[1], held=AT[2], table=AT[3], max_pages=4, max_len=8, stock=AT[4], stock_groups=9,
            state=AT[5], T=5, parents=AT[6], max_nodes=4, step_lens=AT[7], q_start=AT[8], slots=AT[9], positions=AT[10], mask=AT[11],
            lens_out=AT[1], held_out=AT[12], state_out=AT[5])
WRITE = dict(rope=ROPE, q=AT[0], ldq=512, q_out=AT[1], ldqo=512, k=AT[2], ldk=128, v=AT[3], ldv=128, slots=AT[4], positions=AT[5], T=5)
TREE = dict(q=AT[0], ldq=512, table=AT[1], max_pages=4, q_start=AT[2], lens=AT[3], n_seq=3, T=5, mask=AT[4], max_nodes=4, max_len=8,
            scale=0.125, out=AT[5], ldo=512, workspace=AT[6], workspace_bytes=1 << 29)
KEEP = dict(layers=2, n_seq=3, table=AT[0], max_pages=4, q_start=AT[1], lens=AT[2], T=5, tokens=AT[3], targets=AT[4], parents=AT[5],
            max_nodes=4, lens_out=AT[6], path=AT[7], n_path=AT[8], next=AT[9])
CALLS = {"plan": (rg.lora_kv_plan, PLAN), "write": (rg.lora_kv_write_rope, WRITE), "tree": (rg.lora_kv_attend_tree, TREE),
         "accept": (rg.lora_kv_accept, KEEP)}


def _call(which, layout=L, pool=POOL.handle, **change):
    fn, args = CALLS[which]
    return fn(pool, layout, **dict(args, **change), stream=0, check=False)


@pytest.mark.parametrize("which", list(CALLS))
def test_good_arguments_reach_the_last_check(which):
    assert _call(which) == rg.LORA_EINVAL and "bookkeeping-only" in rg.lora_last_error()


@pytest.mark.parametrize("which,change", [
    ("plan", dict(parents=None, mask=None, max_nodes=0)), ("plan", dict(T=0, slots=None, positions=None, parents=None, mask=None)),
    ("plan", dict(lens_out=AT[13], state_out=AT[14])), ("write", dict(q=None, q_out=None)), ("write", dict(q_out=AT[0])),
    ("write", dict(q=AT[0], q_out=AT[0], ldq=768, ldqo=768, k=AT[0] + 1024, ldk=768, v=AT[0] + 1280, ldv=768)),   # one matrix, in place
    ("write", dict(q=AT[0], q_out=AT[2] + 256, ldqo=768, k=AT[2], ldk=768, v=AT[2] + 1280, ldv=768)),
    ("write", dict(rope=rg.lora_rope_t(AT[20], 1, 16, rg.LORA_ROPE_NEIGHBOURS))), ("tree", dict(max_nodes=256)),
    ("tree", dict(max_nodes=1, max_len=1)), ("accept", dict(max_nodes=256)),
    ("accept", dict(T=0, tokens=None, targets=None, parents=None))])
def test_other_good_arguments(which, change):
    assert _call(which, **change) == rg.LORA_EINVAL and "bookkeeping-only" in rg.lora_last_error()


@pytest.mark.parametrize("which", list(CALLS))
@pytest.mark.parametrize("layout", [(0, 1, 64, 1), (8, 3, 64, 1), (8, 2, 96, 1), (8, 2, 64, 0), (8, 2, 64, 3), (1025, 1, 64, 1), (2, 2, 64, 257)])
def test_layouts_refused(which, layout):
    assert _call(which, layout=rg.lora_kv_layout_t(*layout)) == rg.LORA_EINVAL and "layout" in rg.lora_last_error()


REFUSED = [
    ("plan", dict(layers=0)), ("plan", dict(layers=65536)), ("plan", dict(n_seq=-1)), ("plan", dict(n_seq=65536)), ("plan", dict(max_pages=0)),
    ("plan", dict(max_pages=(1 << 21) + 1)), ("plan", dict(max_len=0)), ("plan", dict(max_len=9)), ("plan", dict(stock_groups=0)),
    ("plan", dict(stock_groups=1 << 30)), ("plan", dict(T=-1)), ("plan", dict(T=(1 << 22) + 1)), ("plan", dict(parents=None)),
    ("plan", dict(mask=None)), ("plan", dict(max_nodes=0)), ("plan", dict(max_nodes=257)), ("plan", dict(slots=AT[9] + 4)),
    ("plan", dict(mask=AT[11] + 4)), ("plan", dict(lens_out=AT[1] + 4)), ("plan", dict(lens_out=AT[2])), ("plan", dict(held_out=AT[1])),
    ("plan", dict(state_out=AT[5] + 4)), ("plan", dict(step_lens=AT[1])), ("plan", dict(stock=AT[3] + 64)), ("plan", dict(q_start=AT[7] + 8)),
    ("plan", dict(positions=AT[6])), ("plan", dict(slots=AT[3])), ("plan", dict(slots=None)), ("plan", dict(positions=None)),
    ("write", dict(rope=None)), ("write", dict(rope=rg.lora_rope_t(None, 100, 64, 0))), ("write", dict(rope=rg.lora_rope_t(AT[20] + 4, 100, 64, 0))),
    ("write", dict(rope=rg.lora_rope_t(AT[20], 0, 64, 0))), ("write", dict(rope=rg.lora_rope_t(AT[20], 100, 8, 0))),
    ("write", dict(rope=rg.lora_rope_t(AT[20], 100, 40, 0))), ("write", dict(rope=rg.lora_rope_t(AT[20], 100, 80, 0))),
    ("write", dict(rope=rg.lora_rope_t(AT[20], 100, 64, 2))), ("write", dict(rope=rg.lora_rope_t(AT[20], 100, -16, 0))),
    ("write", dict(q=None)), ("write", dict(q_out=None)), ("write", dict(k=None)), ("write", dict(v=None)), ("write", dict(slots=None)),
    ("write", dict(positions=None)), ("write", dict(slots=AT[4] + 4)), ("write", dict(positions=AT[5] + 2)), ("write", dict(k=AT[2] + 8)),
    ("write", dict(ldq=508)), ("write", dict(ldqo=256)), ("write", dict(ldk=132)), ("write", dict(ldv=64)), ("write", dict(T=-1)),
    ("write", dict(q_out=AT[0] + 16)), ("write", dict(q_out=AT[0], ldqo=520)),
    ("write", dict(q_out=AT[0], k=AT[0], ldk=512)), ("write", dict(q_out=AT[0], v=AT[0], ldv=512)), ("write", dict(T=1, q_out=AT[0], k=AT[0])), ("write", dict(q_out=AT[2])), ("write", dict(q_out=AT[5] - 1024)),
    ("write", dict(q_out=AT[20])), ("write", dict(q=AT[0], q_out=AT[0], ldq=768, ldqo=768, k=AT[0] + 768, ldk=768)),
    ("tree", dict(q=None)), ("tree", dict(out=None)), ("tree", dict(table=None)), ("tree", dict(lens=None)), ("tree", dict(q_start=None)),
    ("tree", dict(mask=None)), ("tree", dict(mask=AT[4] + 4)), ("tree", dict(max_nodes=0)), ("tree", dict(max_nodes=257)),
    ("tree", dict(max_len=0)), ("tree", dict(max_len=9)), ("tree", dict(max_pages=-1)), ("tree", dict(scale=float("nan"))),
    ("tree", dict(scale=float("inf"))), ("tree", dict(out=AT[0])), ("tree", dict(out=AT[4])), ("tree", dict(q=AT[0] + 2)), ("tree", dict(ldq=511)),
    ("tree", dict(ldo=448)), ("tree", dict(n_seq=-1)), ("tree", dict(T=(1 << 22) + 1)),
    ("tree", dict(n_seq=65535, max_pages=1 << 21, max_len=1 << 20)), ("tree", dict(max_pages=1000, max_len=2000, workspace=None)),
    ("tree", dict(max_pages=1000, max_len=2000, workspace_bytes=8)), ("tree", dict(max_pages=1000, max_len=2000, workspace=AT[6] + 16)),
    ("tree", dict(max_pages=1000, max_len=2000, workspace=AT[0])), ("tree", dict(max_pages=1000, max_len=2000, workspace=AT[5])),
    ("accept", dict(layers=0)), ("accept", dict(n_seq=-1)), ("accept", dict(max_pages=0)), ("accept", dict(T=-1)), ("accept", dict(max_nodes=0)),
    ("accept", dict(max_nodes=257)), ("accept", dict(lens_out=AT[2])), ("accept", dict(path=AT[8] - 8)), ("accept", dict(next=AT[8])),
    ("accept", dict(n_path=AT[0])), ("accept", dict(T=0, next=None)), ("accept", dict(T=0, table=None)), ("accept", dict(tokens=AT[3] + 1)),
] + [("plan", {k: None}) for k in ("counts", "lens", "held", "table", "stock", "state", "step_lens", "q_start", "lens_out", "held_out", "state_out")] \
  + [("plan", {k: AT[15] + 2}) for k in ("counts", "held", "table", "state", "parents", "q_start", "held_out")] \
  + [("accept", {k: None}) for k in ("table", "q_start", "lens", "tokens", "targets", "parents", "lens_out", "path", "n_path", "next")]


@pytest.mark.parametrize("which,change", REFUSED, ids=[f"{w}-{'-'.join(map(str, c))}-{i}" for i, (w, c) in enumerate(REFUSED)])
def test_refused(which, change):
    assert _call(which, **change) == rg.LORA_EINVAL
    assert "bookkeeping-only" not in rg.lora_last_error() and "lora_kv" in rg.lora_last_error()


def test_one_row_has_no_stride():
    """Of a single row the distance to the next means nothing, zero and below included: in place it is q's own, elsewhere apart."""
    for change in (dict(q_out=AT[0], ldq=512, ldqo=0), dict(q_out=AT[0], ldq=-8, ldqo=0), dict(q_out=AT[0] + 1024, ldqo=0)):
        assert _call("write", T=1, **change) == rg.LORA_EINVAL and "bookkeeping-only" in rg.lora_last_error()
    for change in (dict(q_out=AT[0] + 16, ldq=0, ldqo=0), dict(q_out=AT[2], ldk=0, ldqo=0), dict(q_out=AT[3] - 512, ldqo=0, ldv=0)):
        assert _call("write", T=1, **change) == rg.LORA_EINVAL and "overlaps" in rg.lora_last_error()


def test_nothing_to_do_and_null_arguments():
    for which, change in [("plan", dict(n_seq=0)), ("write", dict(T=0)), ("tree", dict(n_seq=0)), ("tree", dict(T=0)), ("accept", dict(n_seq=0))]:
        assert _call(which, **change) == rg.LORA_OK, (which, change)
    for which, (fn, args) in CALLS.items():
        assert _call(which, pool=None) == rg.LORA_EINVAL and "pool is NULL" in rg.lora_last_error()
    null = ctypes.POINTER(rg.lora_kv_layout_t)()
    assert rg._lib.lora_kv_attend_tree_workspace_size(POOL.handle, null, 3, 4, 8) == 0


def test_workspace_of_the_largest_call_serves_them_all():
    """Never less for more sequences, nodes or tokens; 0 out of range."""
    size = rg.lora_kv_attend_tree_workspace_size
    for layout in ((4, 4, 64, 1), (4, 1, 64, 1), (2, 2, 128, 1), (1, 1, 256, 1), (32, 1, 64, 1)):
        for dtype in (rg.LORA_BF16, rg.LORA_F32):
            pool = rg.Pool(64, 256, dtype, max_rank=1, device=None)
            lay = rg.lora_kv_layout_t(*layout)
            seqs, nodes, lens = [1, 2, 3, 8, 31, 64, 65, 300, 4000], [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 256], [1, 31, 32, 33, 500, 1024, 1025, 5000, 10 ** 6]
            got = {k: size(pool.handle, lay, *k) for k in itertools.product(seqs, nodes, lens)}
            for s, m, n in got:
                for key in ((s + 1, m, n), (s, m + 1, n), (s, m, n + 1)):
                    larger = min((k for k in got if all(a >= b for a, b in zip(k, key))), default=None)
                    if larger:
                        assert got[s, m, n] <= got[larger], ((s, m, n), larger)
    lay = rg.lora_kv_layout_t(4, 4, 64, 1)
    for bad in ((0, 4, 8), (3, 0, 8), (3, 257, 8), (3, 4, 0), (3, 4, (1 << 22) + 1), (65535, 4, 1 << 20)):
        assert size(POOL.handle, lay, *bad) == 0


def test_plain_forms():
    """A plan, a mask and a path worked out by hand."""
    table, stock = np.full((1, 2, 2, 4), -1, np.int32), np.arange(10, dtype=np.int32).reshape(5, 1, 2)
    table[0, 0, :, 0] = 20, 21
    table[0, 1, :, :2] = [[22, 24], [23, 25]]
    got = draft_ref.plan(1, 2, [3, 0], [1, 2], [1, 2], table, stock, [4, 3, 0, 0], 3, 8, [0, 0, 0], 3)
    assert got["q_start"] == [0, 3, 3] and got["step_lens"] == [4, 0] and got["held"] == [2, 1] and got["lens"] == [4, 2]
    assert got["state"] == [0, 3, 0, 0]                     # group 4 left; sequence 1's second page came behind 4, 0, 1
    assert got["slots"][0].tolist() == [[41, 16, 17], [43, 18, 19]] and got["positions"].tolist() == [1, 2, 2]
    assert got["stock"][2].tolist() == [[24, 25]] and got["table"][0, 0, :, 1].tolist() == [8, 9]
    assert got["mask"][:, 0].tolist() == [1, 3, 5] and not got["err"]
    assert draft_ref.mask_rows([0, 0, 1, 0], [4]) == [1, 3, 7, 9]
    assert draft_ref.accept([0, 0, 0, 2, 3], [9, 4, 5, 6, 7], [5, 0, 6, 8, 0], 5, 0) == [0, 2, 3]
