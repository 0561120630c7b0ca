"""Steps of drafted tokens, call by call: sequences that sit a step out, paths over pages outside the pool, steps without
sequences.  What is expected is written out by hand or worked out beside the call."""
import numpy as np
import pytest
import torch

import rank_gemm_unified_amd as rg
from test_gpu_draft import GEO, Steps, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def plan(s, counts, T=None, in_place=False, **kw):
    """A plan of a Steps' tables; returns it with the changed table and stock."""
    table, stock, lens, held, state = dev(s.table), dev(s.stock), dev(s.lens), dev(s.held), dev(s.state)
    T, out = sum(counts) if T is None else T, None
    if in_place:
        z = dict(dtype=torch.int32, device="cuda")
        out = rg.KvPlan(torch.empty(s.n, **z), torch.empty(s.n + 1, **z), torch.empty((s.layers, 2, T), dtype=torch.int64, device="cuda"),
                        torch.empty(T, **z), None, lens, held, state)
    got = s.pool.kv_plan(s.layout, dev(counts), lens, held, table, stock, state, T, out=out, **kw)
    return got, table.cpu().numpy(), stock.cpu().numpy()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layers", [1, 40])
def test_a_sequence_that_does_not_fit_keeps_its_pages(layers, in_place):
    """Four tokens in six pages of two: two of them are needed.  Over max_len, or behind T, the sequence is refused, and all six
    stay with it; in a step that it takes part in four go back."""
    for kw, counts in ((dict(max_len=6), [1, 3, 0, 1]), (dict(T=3), [1, 3, 0, 1])):
        s = Steps(2, layers, [4, 4, 3, 6], [2, 6, 4, 3], 7, head=3)
        got, table, stock = plan(s, counts, in_place=in_place, **kw)
        assert rg.lora_check_device_errors(s.pool.handle, check=False) == rg.LORA_EDEVICE
        assert got.lens.tolist() == [5, 4, 3, 6] and got.step_lens.tolist() == [5, 0, 0, 0], kw     # (sequence 3 does not fit either)
        # sequence 0 takes a page, sequence 2, without new tokens, gives two back, sequence 1 none
        assert got.held.tolist() == [3, 6, 2, 3] and got.state.tolist() == [4, 8, 2, 0]
        assert np.array_equal(table[:, 1], s.table[:, 1]) and np.array_equal(table[:, 3], s.table[:, 3])
        groups = len(s.stock)
        back = [stock[(3 + 7 + i) % groups] for i in range(2)]
        assert np.array_equal(np.stack(back), s.table[:, 2, :, 2:4].transpose(2, 0, 1))
        rest = [i for i in range(groups) if i not in ((3 + 7) % groups, (3 + 8) % groups)]
        assert np.array_equal(stock[rest], s.stock[rest])
        assert (got.slots[:, :, 1:] == -1).all() and (got.slots[:, :, 0] >= 0).all()
        # the next step has room: the pages that are too many go
        s.table, s.stock, s.lens, s.held, s.state = table, stock, got.lens.tolist(), got.held.tolist(), got.state.tolist()
        got, *_ = plan(s, [0, 1, 0, 0], in_place=in_place)
        assert got.held.tolist() == [3, 3, 2, 3] and got.lens.tolist() == [5, 5, 3, 6] and got.state.tolist() == [4, 11, 0, 0]
        assert rg.lora_check_device_errors(s.pool.handle, check=False) == rg.LORA_OK


@pytest.mark.parametrize("T", [0, 5, 700])
@pytest.mark.parametrize("trees", [False, True])
def test_a_step_without_sequences(T, trees):
    """Every row is behind the last: it has no slot, and the state is the one that came in."""
    lay, z = rg.lora_kv_layout_t(2, 1, 64, 2), dict(dtype=torch.int32, device="cuda")
    pool = rg.Pool(64, 128, rg.LORA_BF16, max_rank=1)
    stock, state, none = dev(np.arange(64).reshape(16, 2, 2)), dev([3, 9, 0, 0]), torch.empty(0, **z)
    for in_place in (False, True):
        out = rg.KvPlan(torch.empty(0, **z), torch.full((1,), 7, **z), torch.full((2, 2, T), 7, dtype=torch.int64, device="cuda"),
                        torch.full((T,), 7, **z), torch.full((T, 1), 7, dtype=torch.int64, device="cuda") if trees else None,
                        none, none, state if in_place else torch.full((4,), 7, **z))
        got = pool.kv_plan(lay, none, none, none, torch.empty((2, 0, 2, 4), **z), stock, state, T, parents=torch.zeros(T, **z) if trees else None,
                           max_nodes=8 if trees else 0, out=out)
        assert (got.slots == -1).all() and (got.positions == 0).all() and got.q_start.tolist() == [0] and got.state.tolist() == [3, 9, 0, 0]
        assert not trees or (got.mask == 0).all()
    assert torch.equal(stock.flatten(), torch.arange(64, **z)) and rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_OK
    for call in (dict(lens=None), dict(q_start=None), dict(state=None)):                # without sequences their lengths may be NULL
        args = dict(layers=2, n_seq=0, counts=None, lens=None, held=None, table=None, max_pages=4, max_len=8, stock=stock, stock_groups=16,
                    state=state, T=0, parents=None, max_nodes=0, step_lens=None, q_start=dev([7]), slots=None, positions=None, mask=None,
                    lens_out=None, held_out=None, state_out=state)
        rc = rg.lora_kv_plan(pool.handle, lay, **{**args, **call}, check=False)
        assert (rc == rg.LORA_OK) == ("lens" in call)


@pytest.mark.parametrize("bad", [64, 2 ** 31 - 1, -1, -2 ** 31])
@pytest.mark.parametrize("place", [3, 1])                   # of the move from place 3 to 2: its source; of 2 to 1: its destination
@pytest.mark.parametrize("geo", ["mha64", "group16"])
def test_moves_from_and_to_a_page_outside_the_pool(geo, place, bad):
    """Two trees whose paths are 0, 2, 3, in two layers.  One page id, of V of one layer of the second tree, lies outside: that one
    move does not happen and is recorded, and every other does.  No other number is bad."""
    nh, nkv, dim, H, tpp = GEO[geo]
    assert tpp == 1                                         # every place has a page of its own
    lay = rg.lora_kv_layout_t(nh, nkv, dim, tpp)
    pool = rg.Pool(64, H, rg.LORA_BF16, max_rank=1)
    table = np.random.default_rng(1).permutation(64).astype(np.int32)[:48].reshape(2, 2, 2, 6)
    parents, tokens, targets = [0, 0, 0, 2], [9, 5, 6, 7], [6, 0, 7, 8]
    old, numbers = [0, 2], [dev(x * 2) for x in (tokens, targets, parents)]
    for hurt in (False, True):
        pool.pages.normal_(generator=torch.Generator(device="cuda").manual_seed(3))
        want, tab = pool.pages.clone(), table.copy()
        if hurt:
            tab[1, 1, 1, old[1] + place] = bad
        for layer in range(2):
            for b in range(2):
                for r in range(2):
                    for at, to in ((2, 1), (3, 2)):
                        if hurt and (layer, b, r) == (1, 1, 1) and place in (at, to):
                            continue
                        w = nkv * dim
                        want[int(table[layer, b, r, old[b] + to]), :w] = want[int(table[layer, b, r, old[b] + at]), :w].clone()
        z = dict(dtype=torch.int32, device="cuda")
        out = rg.KvAccepted(torch.zeros(2, **z), torch.zeros((2, 4), **z), torch.zeros(2, **z), torch.zeros(2, **z))
        got = pool.kv_accept(lay, dev(tab), dev([4, 6]), dev([0, 4, 8]), *numbers, 4, out=out)
        assert got.path.tolist() == [[0, 2, 3, -1]] * 2 and got.lens.tolist() == [3, 5] and got.next.tolist() == [8, 8]
        assert rg.lora_check_device_errors(pool.handle, check=False) == (rg.LORA_EDEVICE if hurt else rg.LORA_OK)
        assert not hurt or "page-id" in rg.lora_last_error()
        assert torch.equal(pool.pages, want)


@pytest.mark.parametrize("given", [False, True])            # on a stream that is given, which is not the current one
def test_lengths_of_sequences_that_sit_a_step_out(given):
    """Plan, acceptance into new tensors, plan: one sequence rests, one finds no free page, one does not fit.  Their lengths and
    pages are what they were, and no group is lost."""
    s = Steps(2, 2, [4, 5, 8, 6], [2, 3, 4, 3], 1, head=2)
    table, stock = dev(s.table), dev(s.stock)
    stream = torch.cuda.Stream() if given else None
    counts, T = [3, 0, 5, 2], 10
    numbers = [dev(x) for x in ([1] * T, [1] * T, [0, 0, 1, 0, 0, 1, 2, 3, 0, 0])]
    args = dict(max_len=12, max_nodes=5, stream=stream)
    torch.cuda.synchronize()
    p = s.pool.kv_plan(s.layout, dev(counts), dev(s.lens), dev(s.held), table, stock, dev(s.state), T, parents=numbers[2], **args)
    torch.cuda.synchronize()
    assert p.step_lens.tolist() == [0, 0, 0, 0] and p.state.tolist()[1:3] == [1, 3]      # two pages, one free: nobody is served
    assert rg.lora_check_device_errors(s.pool.handle, check=False) == rg.LORA_EDEVICE    # (8 and 5 are over 12)
    counts, T = [1, 0, 5, 2], 8
    numbers = [dev(x) for x in ([1] * T, [1] * T, [0, 0, 0, 1, 2, 3, 0, 0])]
    p = s.pool.kv_plan(s.layout, dev(counts), p.lens, p.held, table, stock, p.state, T, parents=numbers[2], **args)
    kept = s.pool.kv_accept(s.layout, table, p.step_lens, p.q_start, *numbers, 5, stream=stream, cached=p.lens)
    again = s.pool.kv_plan(s.layout, dev([0] * 4), kept.lens, p.held, table, stock, p.state, 0, max_len=12, stream=stream)
    torch.cuda.synchronize()
    assert p.step_lens.tolist() == [5, 0, 0, 0] and kept.n_path.tolist() == [1, 0, 0, 0]
    assert kept.lens.tolist() == again.lens.tolist() == [5, 5, 8, 6] and again.held.tolist() == [3, 3, 4, 3] and again.state.tolist()[1] == 0
    assert np.array_equal(table.cpu().numpy()[:, 1:], s.table[:, 1:])
    call = lambda **kw: s.pool.kv_accept(s.layout, table, p.step_lens, p.q_start, *numbers, 5, **kw)  # noqa: E731
    for kw in (dict(cached=p.lens[:3]), dict(cached=p.lens.long()), dict(cached=p.lens.cpu()), dict(cached=p.lens, out=kept)):
        with pytest.raises(ValueError, match="cached"):
            call(**kw)
