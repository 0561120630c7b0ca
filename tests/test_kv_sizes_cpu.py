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
