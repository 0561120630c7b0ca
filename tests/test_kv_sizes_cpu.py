"""Workspace sizes and refusals of the KV-cache calls, on the host."""
import pytest

import rank_gemm_unified_amd as rg


def _sizes(dtype, layout, scores):
    pool = rg.Pool(8, 32768, dtype, max_rank=1, device=None)
    lay = rg.lora_kv_layout_t(*layout)
    return lambda n, m: rg.lora_kv_attend_workspace_size(pool.handle, lay, n, m, scores), pool


@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("dtype", [rg.LORA_BF16, rg.LORA_F32])
@pytest.mark.parametrize("layout", [(32, 8, 128, 1), (32, 32, 128, 1), (4, 1, 64, 1), (40, 2, 64, 1), (8, 2, 256, 4), (64, 64, 64, 1),
                                    (96, 96, 64, 1), (16, 1, 128, 3)])
def test_one_token_workspace_of_the_largest_call_serves_all(layout, dtype, scores):
    """Never less for more sequences or tokens, with scores or without."""
    size, pool = _sizes(dtype, layout, scores)
    lengths = sorted({*range(1, 1101, 13), 96, 97, 191, 192, 193, 255, 256, 257, 384, 385, 511, 512, 513, 767, 768, 769, 1024, 1025, 5000})
    before = [0] * len(lengths)
    for n in [*range(1, 66), 127, 128, 129, 255, 256, 257, 300]:
        got = [size(n, m) for m in lengths]
        assert got == sorted(got), n
        assert all(a <= b for a, b in zip(before, got)), n
        before = got
    if scores:
        without, _ = _sizes(dtype, layout, False)
        assert all(without(n, m) <= size(n, m) for n in (1, 4, 64) for m in lengths)


def test_the_largest_batchs_workspace_serves_a_smaller_one():
    """A workspace sized for 32 sequences is enough for 4 of the same length."""
    size, pool = _sizes(rg.LORA_BF16, (32, 8, 128, 1), False)
    assert 0 < size(4, 1024) <= size(32, 1024)
    assert size(1, 512) == size(32, 200) == 0        # one launch, for every smaller call too: none is needed


# ---- what is written overlaps nothing else (addresses that are never read: every call is refused) ----------
A, GAP = 1 << 40, 1 << 30
POOL = rg.Pool(64, 256, rg.LORA_BF16, max_rank=1, device=None)
LAYOUT = rg.lora_kv_layout_t(8, 2, 64, 2)
ATTEND = dict(q=A, ldq=512, table=A + GAP, max_pages=300, lens=A + 2 * GAP, n_seq=3, max_len=600, scale=0.125, out=A + 3 * GAP,
              ldo=512, prior=A + 4 * GAP, scores=A + 5 * GAP, workspace=A + 6 * GAP, workspace_bytes=1 << 29)
STARTS = A + 7 * GAP


@pytest.mark.parametrize("chunk", [False, True])
@pytest.mark.parametrize("written,ends_at", [(w, b) for w in ("out", "scores", "workspace")
                                             for b in ("q", "table", "lens", "q_start", "prior", "out", "scores", "workspace") if b != w])
def test_what_is_written_overlaps_nothing(written, ends_at, chunk):
    if ends_at == "q_start" and not chunk:
        pytest.skip("no row ranges")
    args = dict(ATTEND, **(dict(q_start=STARTS, T=5) if chunk else {}))
    call = rg.lora_kv_attend_chunk if chunk else rg.lora_kv_attend
    rows = 5 if chunk else 3
    need = (rg.lora_kv_attend_chunk_workspace_size(POOL.handle, LAYOUT, 3, 5, 600, True) if chunk
            else rg.lora_kv_attend_workspace_size(POOL.handle, LAYOUT, 3, 600, True))
    size = {"q": rows * 1024, "out": rows * 1024, "table": 3 * 2 * 300 * 4, "lens": 12, "q_start": 16, "prior": 3 * 600 * 4,
            "scores": 3 * 600 * 4, "workspace": need}
    step = {"out": 16, "scores": 4, "workspace": 256}[written]
    end = args[ends_at] + size[ends_at]
    inside, behind = (end - 1) // step * step, -(-end // step) * step
    assert call(POOL.handle, LAYOUT, **dict(args, **{written: inside}), stream=0, check=False) == rg.LORA_EINVAL
    assert "overlap" in rg.lora_last_error()
    assert call(POOL.handle, LAYOUT, **dict(args, **{written: behind}), stream=0, check=False) == rg.LORA_EINVAL
    assert "bookkeeping-only" in rg.lora_last_error()
    before = args[ends_at] - size[written]
    assert call(POOL.handle, LAYOUT, **dict(args, **{written: before // step * step}), stream=0, check=False) == rg.LORA_EINVAL
    assert "bookkeeping-only" in rg.lora_last_error()


@pytest.mark.parametrize("chunk", [False, True])
def test_scores_may_be_their_own_prior(chunk):
    args = dict(ATTEND, prior=ATTEND["scores"], **(dict(q_start=STARTS, T=5) if chunk else {}))
    (rg.lora_kv_attend_chunk if chunk else rg.lora_kv_attend)(POOL.handle, LAYOUT, **args, stream=0, check=False)
    assert "bookkeeping-only" in rg.lora_last_error()
