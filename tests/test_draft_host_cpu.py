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
