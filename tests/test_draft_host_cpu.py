"""What the calls of a step of drafted tokens, and the KV calls before them, refuse on the host."""
import pytest
import torch

import rank_gemm_unified_amd as rg

L = rg.lora_kv_layout_t(4, 2, 64, 1)


def test_a_pool_on_the_host_takes_no_call(monkeypatch):
    """Tensors on the host are no device memory, also where the pool's pages lie there."""
    monkeypatch.setattr(rg, "lora_pool_create", lambda *a: None)
    pool = rg.Pool(8, 128, rg.LORA_BF16, max_rank=1, device="cpu")
    i32 = dict(dtype=torch.int32)
    rows = lambda w: torch.zeros((2, w), dtype=torch.bfloat16)  # noqa: E731
    table, one, start = torch.zeros((2, 2, 1), **i32), torch.ones(2, **i32), torch.arange(3, **i32)
    for call in (lambda: pool.kv_write(L, rows(128), rows(128), table, one),
                 lambda: pool.kv_attend(L, rows(256), table, one),
                 lambda: pool.kv_attend_tree(L, rows(256), table, one, start, torch.ones((2, 1), dtype=torch.int64)),
                 lambda: pool.kv_write_rope(L, None, None, rows(128), rows(128), torch.zeros((2, 2), dtype=torch.int64), one),
                 lambda: pool.kv_plan(L, one, one, one, table[None], torch.zeros((4, 1, 2), **i32), torch.zeros(4, **i32), 2),
                 lambda: pool.kv_accept(L, table[None], one, start, one, one, one, 1)):
        with pytest.raises(ValueError, match="is wanted|are wanted"):
            call()


@pytest.mark.parametrize("dtype", [rg.LORA_BF16, rg.LORA_F32])
@pytest.mark.parametrize("layout", [(514, 514, 64, 1), (768, 768, 64, 1), (1022, 1022, 64, 1), (1024, 512, 64, 1), (1024, 1024, 64, 1),
                                    (600, 600, 64, 1), (512, 512, 128, 1), (900, 300, 64, 1), (511, 511, 64, 1), (130, 130, 256, 1), (40, 40, 128, 1), (40, 8, 128, 5)])
def test_a_tree_workspace_serves_every_smaller_call(layout, dtype):
    """Never less for more sequences, nodes or tokens, up to the most heads: each size against the next larger ones."""
    pool = rg.Pool(8, layout[1] * layout[2] * layout[3], dtype, max_rank=1, device=None)
    lay, size = rg.lora_kv_layout_t(*layout), rg.lora_kv_attend_tree_workspace_size
    seqs, nodes = [1, 2, 3, 4, 8, 31, 64, 65, 300, 4000], [1, 5, 6, 8, 9, 16, 17, 21, 22, 32, 33, 64, 65, 85, 86, 128, 129, 256]
    lens = [1, 31, 32, 33, 64, 65, 256, 257, 512, 513, 1024, 1025, 2048, 2049, 5000, 10 ** 6]
    got = {(i, j, k): size(pool.handle, lay, s, m, n) for i, s in enumerate(seqs) for j, m in enumerate(nodes) for k, n in enumerate(lens)}
    for (i, j, k), n in got.items():
        for more in ((i + 1, j, k), (i, j + 1, k), (i, j, k + 1)):
            assert n <= got.get(more, n), (seqs[i], nodes[j], lens[k], more)


def test_rows_that_finish():
    """Numbers on the host that are no row are refused before anything changes."""
    cache = object.__new__(rg.KvDraftCache)
    cache.max_seqs, cache.step, cache.lens = 3, None, torch.tensor([4, 5, 6], dtype=torch.int32)
    for bad in ([3], [0, -1], torch.tensor([1, 2 ** 40]), 7):
        with pytest.raises(ValueError, match="not in"):
            cache.finish(bad)
        assert cache.lens.tolist() == [4, 5, 6]
    cache.finish([])
    assert cache.lens.tolist() == [4, 5, 6]
    cache.finish([2, 0, 2])
    assert cache.lens.tolist() == [0, 5, 0]
