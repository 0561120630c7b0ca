"""Rounding, zero weights and values that are not finite in the KV-cache attention calls, on the device."""
import numpy as np
import pytest
import torch

from test_gpu_kv import Case, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("geo,n,at", [
    ("gqa64", 200, 100), ("mqa128", 200, 64), ("dim256", 300, 70), ("group3", 200, 130),
    ("gqa64", 1100, 100), ("gqa64", 1100, 700), ("mqa128", 900, 100),       # in ranges
    ("wide64", 200, 100), ("wide64_kv64", 260, 64),                         # in pairs
])
def test_a_chunks_largest_weight_is_not_rounded(geo, n, at):
    """A row's largest weight is one, whatever smaller maximum the tokens before it had.  Token 0 has logit 0 and
    values 0, token `at` logit c / 8 and values 1, the others no weight to speak of: out = 1 / (1 + exp(-c / 8)).
    Only the output's own rounding is left, half a step of 2^-8 in [1/2, 1) and of 2^-7 at 1, and the float32 sums
    (1e-5 is 80 of their steps)."""
    rows = 44 if geo.startswith(("gqa", "mqa", "dim", "group")) else 128
    c = Case(geo, "bf16", [n] * (1 if rows == 44 else 4), [rows] * (1 if rows == 44 else 4))
    tpp, dim, w = c.layout.tokens_per_page, c.layout.head_dim, c.layout.n_kv_heads * c.layout.head_dim
    c.pool.pages.zero_()
    held = c.pool.pages[:, : tpp * w].view(-1, tpp, c.layout.n_kv_heads, dim)
    for b in range(c.n):
        ids = [torch.as_tensor(c.table[b, r, np.arange(n) // tpp].astype(np.int64), device="cuda") for r in range(2)]
        slot = torch.arange(n, device="cuda") % tpp
        held[ids[0], slot, :, 0] = -1000.0
        held[ids[0][0], slot[0], :, 0] = 0.0
        held[ids[0][at], slot[at], :, 0] = 1.0
        held[ids[1][at], slot[at]] = 1.0
    step = torch.arange(rows, device="cuda") % 44 + 1                       # logits of 1/8 to 44/8
    c.q.zero_()
    c.q.view(c.n, rows, -1, dim)[..., 0] = step[None, :, None].to(c.dt)
    out = c.run(scale=0.125)
    assert c.errors() == 0
    want = 1 / (1 + torch.exp(-step.double() / 8))
    want[torch.arange(n - rows, n, device="cuda") < at] = 0                 # rows before that token
    off = (out.view(c.n, rows, -1).double() - want[None, :, None]).abs()
    assert (off <= 2.0 ** -9 + 1e-5).all(), (off.max().item(), off.amax((0, 2)).topk(3))


def _all_minus_infinity(c, b):
    """Sequence b: every product with a query is -inf, and among the values are infinities and NaN."""
    tpp, dim = c.layout.tokens_per_page, c.layout.head_dim
    held = c.pool.pages[:, : tpp * c.layout.n_kv_heads * dim].view(-1, tpp, c.layout.n_kv_heads, dim)
    n = c.lens[b]
    ids = [torch.as_tensor(c.table[b, r, np.arange(n) // tpp].astype(np.int64), device="cuda") for r in range(2)]
    slot = torch.arange(n, device="cuda") % tpp
    held[ids[0], slot, :, 0] = -float("inf")
    c.q.view(c.T, -1, dim)[..., 0] = 1.0
    for at, x in ((0, float("inf")), (n // 2, -float("inf")), (n - 1, float("nan"))):
        held[ids[1][at], slot[at]] = x


def _zero_rows(geo, dtype, lens, new, scores):
    c = Case(geo, dtype, lens, new, seed=21)
    _all_minus_infinity(c, 1)
    prior = torch.rand((c.n, c.cap), device="cuda") if scores else None
    sc = torch.full((c.n, c.cap), -3.0, device="cuda") if scores else None
    out = c.run(scores=sc, prior=prior)
    rows = slice(1, 2) if new is None else slice(new[0], new[0] + new[1])
    assert (out[rows] == 0).all()
    assert torch.isfinite(out).all() and (out[: rows.start] != 0).any() and (out[rows.stop:] != 0).any()
    if scores:
        n = c.lens[1]
        assert torch.equal(sc[1, :n], prior[1, :n]) and (sc[1, n:] == -3.0).all()
    assert c.errors() == 0


@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("geo,lens", [
    ("gqa64", [40, 33, 50]), ("mqa128", [90, 64, 31]), ("dim256", [40, 65, 50]),               # one launch without scores
    ("mha128", [1500, 1, 1500]), ("mqa128", [70] * 300), ("group20", [700, 64, 900]),           # whole in one range, and pieces
    ("gqa64", [2000, 1500, 3000]), ("dim256", [2000, 1500, 300]), ("gqa64", [900] * 60),        # many pieces, and few
])
def test_a_token_no_weight_reaches_is_zero(geo, lens, dtype, scores):
    """Where every product is -inf the output is zero, whatever the values hold."""
    _zero_rows(geo, dtype, lens, None, scores)


@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("geo,lens,new", [
    ("gqa64", [90, 80, 50], [90, 80, 50]), ("mqa128", [200, 150, 70], [20, 33, 70]), ("dim256", [60, 130, 40], [3, 130, 40]),
    ("gqa64", [900, 1500, 300], [3, 20, 9]), ("dim256", [900, 700, 300], [3, 20, 9]),           # in ranges
    ("wide64", [300, 257, 200], [300, 257, 200]),                                               # in pairs
])
def test_a_chunk_no_weight_reaches_is_zero(geo, lens, new, dtype, scores):
    _zero_rows(geo, dtype, lens, new, scores)


@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("geo,lens", [("gqa64", [40, 133]), ("mqa128", [90, 64]), ("dim256", [40, 65]), ("gqa64", [2000, 1500])])
def test_a_weight_of_zero_adds_nothing(geo, lens, dtype, scores):
    """The largest finite values meet weights that are zero (a product of -inf, or one 200 below the others) and one of
    exp(-80): what they add is their weight times them.  Token 1: -inf, token 2: -200, token 3: exp(-80), the others 0."""
    c = Case(geo, dtype, lens, seed=22)
    tpp, dim = c.layout.tokens_per_page, c.layout.head_dim
    held = c.pool.pages[:, : tpp * c.layout.n_kv_heads * dim].view(-1, tpp, c.layout.n_kv_heads, dim)
    big = 2.0 ** 127
    c.q.zero_()
    c.q.view(c.T, -1, dim)[..., 0] = 1.0
    for b, n in enumerate(lens):
        ids = [torch.as_tensor(c.table[b, r, np.arange(n) // tpp].astype(np.int64), device="cuda") for r in range(2)]
        slot = torch.arange(n, device="cuda") % tpp
        held[ids[0], slot] = 0.0
        held[ids[1], slot] = 1.0
        for t, x in ((1, -float("inf")), (2, -200.0), (3, -80.0)):
            held[ids[0][t], slot[t], :, 0] = x
            held[ids[1][t], slot[t], :, 7 + t] = big
    sc = torch.zeros((c.n, c.cap), device="cuda") if scores else None
    out = c.run(scale=1.0, scores=sc).view(c.n, -1, dim).double()
    for b, n in enumerate(lens):
        want = torch.full((dim,), (n - 3.0) / (n - 3.0), dtype=torch.float64, device="cuda")
        want[10] += np.exp(-80.0) * big / (n - 3.0)
        # half a step of the output (2^-8), the weight's two parts (2^-15), and exp(-80) from a logit that float32 holds
        # to half a step of 115 in base 2 (2^-18 * ln 2)
        assert ((out[b] - want).abs() <= want * (2.0 ** -8 + 2.0 ** -14 + 2.0 ** -17)).all(), (b, out[b, 0, 7:12], want[7:12])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("geo,lens", [("gqa64", [40, 133]), ("mqa128", [90, 64]), ("dim256", [40, 65]), ("gqa64", [2000, 1500])])
def test_a_weight_of_zero_times_infinity_is_not_a_number(geo, lens, dtype):
    c = Case(geo, dtype, lens, seed=23)
    tpp, dim = c.layout.tokens_per_page, c.layout.head_dim
    held = c.pool.pages[:, : tpp * c.layout.n_kv_heads * dim].view(-1, tpp, c.layout.n_kv_heads, dim)
    c.q.view(c.T, -1, dim)[..., 0] = 1.0
    for b in range(c.n):
        k, v = (int(c.table[b, r, 17 // tpp]) for r in range(2))
        held[k, 17 % tpp, :, 0] = -float("inf")
        held[v, 17 % tpp, :, 5] = float("inf")
    for sc in (None, torch.zeros((c.n, c.cap), device="cuda")):
        out = c.run(scores=sc).view(c.n, -1, dim)
        assert torch.isnan(out[..., 5]).all()
        out[..., 5] = 0
        assert torch.isfinite(out).all()
