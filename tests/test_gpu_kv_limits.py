"""The KV-cache calls at the largest sizes that their description allows, on the device."""
import numpy as np
import pytest
import torch

import kv_ref
import rank_gemm_unified_amd as rg
from gpu_helpers import say
from test_gpu_kv import DT, _gpu, close  # noqa: F401

pytestmark = pytest.mark.gpu

LAYOUT = rg.lora_kv_layout_t(1, 1, 64, 1)
MOST, LONGEST = rg.LORA_MAX_SEQS, rg.LORA_MAX_KV_TOKENS


def _pool(pages, dtype, seed):
    pool = rg.Pool(pages, 64, rg.LORA_BF16 if dtype is torch.bfloat16 else rg.LORA_F32, max_rank=1)
    pool.pages.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
    return pool


def _some(n, table, lens, starts, q, out, pool, scores, dtype, scale=0.125):
    """`n` sequences among all, the first and the last of them too, against float64."""
    rng = np.random.default_rng(5)
    for b in sorted({0, 1, len(lens) - 1, *rng.integers(0, len(lens), n).tolist()}):
        rows = slice(b, b + 1) if starts is None else slice(int(starts[b]), int(starts[b + 1]))
        m = rows.stop - rows.start
        want, tol, sw, stol = kv_ref.attend(pool.pages, LAYOUT, q[rows], table[b:b + 1].cpu().numpy(), [int(lens[b])],
                                            None if starts is None else [0, m], scale, kv_ref.ROUNDED[dtype, starts is not None])
        close(out[rows], want, tol, dtype, f"sequence {b}")
        if scores is not None:
            k = int(lens[b])
            close(scores[b:b + 1, :k], sw[:, :k], stol[:, :k], torch.float32, f"scores of {b}")


@pytest.mark.parametrize("dtype", list(DT))
def test_the_most_sequences_of_one_token(dtype):
    dt, width = DT[dtype], 40
    lens = torch.arange(MOST, device="cuda", dtype=torch.int32) % (width + 1)          # 0 to 40 tokens
    pool = _pool(200_000, dt, 61)
    g = torch.Generator(device="cuda").manual_seed(62)
    table = torch.randint(0, 200_000, (MOST, 2, width), generator=g, device="cuda", dtype=torch.int32)
    q = torch.empty((MOST, 64), dtype=dt, device="cuda").normal_(generator=g) * 2
    scores = torch.full((MOST, width), -3.0, device="cuda")
    for sc in (None, scores):
        out = pool.kv_attend(LAYOUT, q, table, lens, scores=sc)
        assert (out[lens == 0] == 0).all()
        _some(40, table, lens.tolist(), None, q, out, pool, sc, dt)
    assert (scores[torch.arange(width, device="cuda") >= lens[:, None]] == -3.0).all()
    assert rg.lora_check_device_errors(pool.handle, check=False) == 0


def test_the_most_sequences_and_rows_of_a_chunk():
    """64 new tokens in each of 65535 sequences: 2^22 rows but 64.  Written, then read."""
    dt, m = torch.bfloat16, 64
    pool = _pool(2 * MOST * m, dt, 63)
    table = torch.arange(2 * MOST * m, device="cuda", dtype=torch.int32).view(MOST, 2, m).flip(0).contiguous()
    lens = torch.full((MOST,), m, device="cuda", dtype=torch.int32)
    starts = torch.arange(MOST + 1, device="cuda", dtype=torch.int32) * m
    T = MOST * m
    assert T <= rg.LORA_MAX_TOKENS
    g = torch.Generator(device="cuda").manual_seed(64)
    k, v, q = (torch.empty((T, 64), dtype=dt, device="cuda").normal_(generator=g) for _ in range(3))
    pool.kv_write(LAYOUT, k, v, table, lens, starts)
    held = pool.pages[table.view(-1).long()].view(MOST, 2, m, 64)
    assert torch.equal(held[:, 0], k.view(MOST, m, 64)) and torch.equal(held[:, 1], v.view(MOST, m, 64))
    del held, k, v
    scores = torch.zeros((MOST, m), device="cuda")
    out = pool.kv_attend_chunk(LAYOUT, q, table, lens, starts, scores=scores)
    _some(30, table, lens.tolist(), starts.tolist(), q, out, pool, scores, dt)
    assert torch.equal(pool.kv_attend_chunk(LAYOUT, q, table, lens, starts), out)
    assert rg.lora_check_device_errors(pool.handle, check=False) == 0


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [None, 3])
def test_the_longest_cache(dtype, rows):
    """2^22 tokens, a few of which, up to the last one, hold most of the weight."""
    dt, n = DT[dtype], LONGEST
    pool = _pool(2 * n, dt, 65)
    table = torch.randperm(2 * n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(66)).to(torch.int32).view(1, 2, n)
    lens = torch.tensor([n], device="cuda", dtype=torch.int32)
    q = torch.ones((rows or 1, 64), dtype=dt, device="cuda")
    for i, t in enumerate((5, n // 2 + 1, n - 2, n - 1)):                              # logits of 16 and more
        pool.pages[int(table[0, 0, t])] = 2.0 + i / 16
        pool.pages[int(table[0, 1, t])] = 1.0 + i
    K, V = (pool.pages[table[0, r].long()].double() for r in range(2))
    x = (K @ q[0].double()) * 0.125
    scores = torch.zeros((1, n), device="cuda")
    if rows is None:
        out = pool.kv_attend(LAYOUT, q, table, lens, scores=scores)
        other = pool.kv_attend(LAYOUT, q, table, lens)
    else:
        starts = torch.tensor([0, rows], device="cuda", dtype=torch.int32)
        out = pool.kv_attend_chunk(LAYOUT, q, table, lens, starts, scores=scores)
        other = pool.kv_attend_chunk(LAYOUT, q, table, lens, starts)
    assert torch.equal(out, other)
    # Sums: a lane adds at most 2^22 / 64 weights of its share one after the other, the pieces add 2048 at most.
    sums = (2 ** 16 + 2048) * kv_ref.EPS32
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    for r in range(rows or 1):
        seen = n - (rows or 1) + 1 + r
        p = torch.softmax(x[:seen], 0)
        total[:seen] += p
        want, size = p @ V[:seen], p @ V[:seen].abs()
        tol = size * (sums + kv_ref.ROUNDED[dt, rows is not None]) + kv_ref.HALF[dt] * want.abs()
        off = (out[r].double() - want).abs()
        say(f"row {r}: {(off / tol).max().item():.3f} of the bound")
        assert (off <= tol).all() and want.abs().min() > 0.1
    assert ((scores[0].double() - total).abs() <= total * (sums + 2 ** -15)).all()      # a logit of 25 is off by 2^-16 at most
    assert rg.lora_check_device_errors(pool.handle, check=False) == 0


def test_eviction_from_the_longest_cache():
    n = LONGEST
    pool = _pool(16, torch.bfloat16, 67)
    g = torch.Generator(device="cuda").manual_seed(68)
    table = torch.randint(0, 1 << 30, (1, 1, 2, n), generator=g, device="cuda", dtype=torch.int32)
    scores = torch.rand((1, 1, n), generator=g, device="cuda")
    lens = torch.tensor([n], device="cuda", dtype=torch.int32)
    drop = 1_000_003
    t, s, ln, gone, count = pool.kv_evict(LAYOUT, table, scores, lens, n - drop, 4, 64)
    assert ln.tolist() == [n - drop] and count.tolist() == [drop]
    free = torch.arange(4, n - 64, device="cuda")
    order = scores[0, 0, free].sort(stable=True).indices                                # ties: the earlier page
    out = torch.zeros(n, dtype=torch.bool, device="cuda")
    out[free[order[:drop]]] = True
    for r in range(2):
        assert torch.equal(t[0, 0, r, : n - drop], table[0, 0, r][~out]) and (t[0, 0, r, n - drop:] == -1).all()
        assert torch.equal(gone[0, 0, r, :drop], table[0, 0, r][out]) and (gone[0, 0, r, drop:] == -1).all()
    assert torch.equal(s[0, 0, : n - drop], scores[0, 0][~out]) and (s[0, 0, n - drop:] == 0).all()
    assert rg.lora_check_device_errors(pool.handle, check=False) == 0
