"""How exact the attention of trees is, whatever the number of rows: the weights enter the product with V as two bfloat16
numbers, off by 2^-15 of themselves at most (kv_ref.ROUNDED), so that rows whose values cancel keep what is left of them."""
import numpy as np
import pytest
import torch

import draft_ref
import kv_ref
from test_gpu_draft import Trees, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def exact(c):
    return draft_ref.attend(c.pool.pages, c.layout, c.q, c.table, c.lens, c.starts, c.bits, c.scale, kv_ref.ROUNDED[c.dt, False])


# Over 16 rows of a K/V head: whole sequences and ranges, one head and two of a workgroup, every head dim, several blocks of rows.
@pytest.mark.parametrize("geo,lens,new", [
    ("mha64", [300, 41, 90], [17, 40, 33]), ("mha64", [1500, 1100], [30, 64]), ("gqa64", [45, 1100], [12, 60]),
    ("mqa128", [2100], [40]), ("group16", [700], [9]), ("dim256", [700, 1100], [16, 9]), ("dim256", [3000], [64]),
    ("kv8", [1990, 2000, 1000, 30, 17, 700, 900, 1600], [16, 9, 16, 9, 16, 13, 10, 16]), ("kv8", [5000], [64]),
    ("mha128", [700, 1010, 33, 900], [17, 40, 33, 64]), ("gqa64", [11 + b % 60 for b in range(512)], [5 + b % 2 for b in range(512)])],
    ids=lambda x: x if isinstance(x, str) else f"{len(x)}x{max(x)}")
def test_weights_of_many_rows(geo, lens, new):
    c = Trees(geo, "bf16", lens, new, seed=21)
    want, tol = exact(c)
    close(c.run(), want, tol, c.dt, geo)


@pytest.mark.parametrize("nodes", [4, 64])
def test_the_same_tree_in_a_call_for_larger_ones(nodes):
    """Trees of four nodes, whatever max_nodes says."""
    c = Trees("mha64", "bf16", [300, 41], [4, 4], seed=22, max_nodes=nodes)
    want, tol = exact(c)
    close(c.run(), want, tol, c.dt, f"max_nodes {nodes}")


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("geo,lens,new", [("mha64", [40, 30], [3, 4]), ("mha64", [60, 70], [20, 33]), ("kv8", [5000], [32]), ("dim256", [90], [33])])
def test_an_infinite_value_of_a_cached_token_stays_that_infinity(geo, lens, new, value):
    """Its weight is not zero (the logits are within a few units of one another): every row is that infinity there."""
    c = Trees(geo, "bf16", lens, new, seed=23)
    c.q *= 0.1
    want, tol = exact(c)
    tpp, dim = c.layout.tokens_per_page, c.layout.head_dim
    group, nkv = c.layout.n_heads // c.layout.n_kv_heads, c.layout.n_kv_heads
    clean = np.ones(want.shape, bool)
    for b, n in enumerate(c.lens):
        t, kvh, d = min(7, n - c.new[b] - 1), b % nkv, 5
        c.pool.pages[int(c.table[b, 1, t // tpp]), (t % tpp * nkv + kvh) * dim + d] = value
        for h in range(kvh * group, (kvh + 1) * group):
            clean[c.starts[b]:c.starts[b + 1], h * dim + d] = False
    out = c.run()
    dirty = torch.as_tensor(~clean, device="cuda")
    assert (out[dirty] == value).all()
    close(torch.where(dirty, 0.0, out), np.where(clean, want, 0), np.where(clean, tol, 0), c.dt, geo)
