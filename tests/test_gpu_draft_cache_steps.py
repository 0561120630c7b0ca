"""KvDraftCache: requests that end inside a step, steps that are captured in parts, paths that are kept once."""
import pytest
import torch

import rank_gemm_unified_amd as rg
from test_gpu_draft import dev

pytestmark = pytest.mark.gpu

LAYOUT, LAYERS = rg.lora_kv_layout_t(4, 2, 64, 2), 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rows(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((T, w), generator=g, device="cuda") for w in (256, 128, 128)]


def make(groups=40, request=7, pool=None):
    pool = pool or rg.Pool(400, 256, rg.LORA_F32, max_rank=1)
    pool.pages.zero_()
    return rg.KvDraftCache(pool, LAYERS, LAYOUT, 3, 60, groups, request, rg.Rope.of(64, 64))


def layers(cache, q, k, v):
    out = []
    for layer in range(LAYERS):
        out.append(cache.attend(layer, cache.write(layer, q, k, v)))
    return out


def pages_are_whole(cache, groups=40):
    """What the lengths need is held, the rest is free, and no group is lost or held twice."""
    cache.plan(dev([0, 0, 0]), 1)
    held = [-(-int(n) // 2) for n in cache.lens]
    head, free = cache.state.tolist()[:2]
    assert cache.held.tolist() == held and free == groups - sum(held)
    ids = [x for i in range(free) for x in cache.stock[(head + i) % groups].flatten().tolist()]
    ids += [x for b in range(3) for e in range(held[b]) for x in cache.table[:, b, :, e].flatten().tolist()]
    assert sorted(ids) == sorted(rg.lora_pool_kv_pages(cache.pool.handle, cache.request))
    assert rg.lora_check_device_errors(cache.pool.handle, check=False) == rg.LORA_OK


PARENTS, TOKENS, TARGETS = [0, 0, 0, 2], [9, 5, 6, 7], [6, 0, 7, 8]      # the path is 0, 2, 3


@pytest.mark.parametrize("when", ["before the layers", "between the layers", "before the acceptance"])
@pytest.mark.parametrize("as_list", [True, False])
def test_a_request_that_ends_inside_a_step_stays_ended(when, as_list):
    cache, other = make(), make()
    numbers = [dev(x * 3) for x in (TOKENS, TARGETS, PARENTS)]
    for c in (cache, other):
        c.plan(dev([5, 7, 6]), 18)
        layers(c, *rows(18, 1))
        c.plan(dev([4, 4, 4]), 12, numbers[2], 4)
    end = lambda: cache.finish([1] if as_list else torch.tensor([1], device="cuda"))  # noqa: E731
    x = rows(12, 2)
    want = layers(other, *x)
    if when == "before the layers":
        end()
        got = layers(cache, *x)
        assert all((g[4:8] == 0).all() for g in got)
    elif when == "between the layers":
        got = [cache.attend(0, cache.write(0, *x))]
        end()
        got.append(cache.attend(1, cache.write(1, *x)))
        assert torch.equal(got[0], want[0]) and (got[1][4:8] == 0).all()
    else:
        got = layers(cache, *x)
        end()
        assert torch.equal(got[1], want[1])
    for g, w in zip(got, want):
        assert torch.equal(g[:4], w[:4]) and torch.equal(g[8:], w[8:])
    kept = cache.accept(*numbers[:2])
    assert cache.lens.tolist() == [8, 0, 9] and kept.n_path.tolist() == [3, 0, 3] and kept.next.tolist() == [8, -1, 8]
    pages_are_whole(cache)
    assert cache.held.tolist() == [4, 0, 5]
    # another request in that row begins at place 0
    cache.plan(dev([0, 3, 0]), 3)
    assert cache.step.positions.tolist() == [0, 1, 2] and cache.lens.tolist() == [8, 3, 9]
    first = cache.attend(0, cache.write(0, *rows(3, 4)))
    assert torch.allclose(first[0].view(4, 64), rows(3, 4)[2][0].view(2, 64).repeat_interleave(2, 0), rtol=2 ** -22, atol=0)


def test_numbers_on_the_device_that_are_no_row_finish_none():
    cache = make()
    cache.plan(dev([5, 7, 6]), 18)
    layers(cache, *rows(18, 1))
    for some in ([], [-1], [3, 2 ** 40, -2 ** 40]):
        cache.finish(torch.tensor(some, dtype=torch.int64, device="cuda"))
    assert cache.lens.tolist() == cache.step.step_lens.tolist() == [5, 7, 6]
    cache.finish(torch.tensor([3, 2, -1, 2], device="cuda"))
    assert cache.lens.tolist() == cache.step.step_lens.tolist() == [5, 7, 0]
    pages_are_whole(cache)


def same(one, two):
    return all(torch.equal(a, b) for a, b in ((one.lens, two.lens), (one.held, two.held), (one.state, two.state), (one.table, two.table),
                                              (one.stock, two.stock), (one.pool.pages, two.pool.pages)))


def trees(seed):
    """Counts, parents, tokens and targets of a step of up to four nodes a sequence, twelve rows."""
    g = torch.Generator().manual_seed(seed)
    counts = torch.randint(1, 5, (3,), generator=g).tolist()
    counts[seed % 3] = 0 if seed % 2 else 4
    fill = [0] * (12 - sum(counts))
    parents = [0 if i == 0 else int(torch.randint(0, i, (1,), generator=g)) for c in counts for i in range(c)] + fill
    return [dev(counts), dev(parents)] + [torch.randint(0, 2, (12,), generator=g).int().cuda() for _ in range(2)]


@pytest.mark.parametrize("inside", ["plan", "plan and layers", "all", "acceptance"])
def test_steps_captured_in_parts(inside):
    """What is captured is replayed step after step, the rest is called between the replays, beside a cache that runs all of it
    eagerly.  A path is kept once: a second acceptance of the same step, called or replayed, moves nothing."""
    cache, other = make(), make()
    for c in (cache, other):
        c.plan(dev([5, 7, 6]), 18)
        layers(c, *rows(18, 1))
    numbers, x = trees(0), rows(12, 2)
    counts, parents, tokens, targets = numbers
    parts = [lambda c: c.plan(counts, 12, parents, 4), lambda c: layers(c, *x), lambda c: c.accept(tokens, targets)]
    upto = {"plan": 1, "plan and layers": 2, "all": 3, "acceptance": 0}[inside]
    before = [t.clone() for t in (cache.lens, cache.held, cache.state, cache.table, cache.stock, cache.pool.pages)]
    side = torch.cuda.Stream()                              # sets the libraries up; what it changes is put back
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for part in parts:
            part(cache)
    torch.cuda.current_stream().wait_stream(side)
    for t, b in zip((cache.lens, cache.held, cache.state, cache.table, cache.stock, cache.pool.pages), before):
        t.copy_(b)
    assert same(cache, other)
    graph = torch.cuda.CUDAGraph()
    if inside != "acceptance":
        with torch.cuda.graph(graph):
            done = [part(cache) for part in parts[:upto]]
        assert same(cache, other)                           # nothing ran yet
    for seed in range(6):
        for t, new in zip(numbers, trees(seed)):
            t.copy_(new)
        for i, t in enumerate(x):
            t.copy_(rows(12, 10 + seed)[i])
        want = [part(other) for part in parts]
        if inside == "acceptance":                          # of one step each, captured behind its layers
            got = [part(cache) for part in parts[:2]]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got.append(parts[2](cache))
            graph.replay()
        else:
            graph.replay()
            got = done + [part(cache) for part in parts[upto:]]
        assert same(cache, other), seed
        kept = [t.clone() for t in got[2]]
        assert all(torch.equal(a, b) for a, b in zip(kept, want[2]))
        there = int(other.step.q_start[-1])                  # (rows behind the last hold anything)
        assert torch.equal(got[1][1][:there], want[1][1][:there])
        torch.randn(100, device="cuda").sum().item()         # the program's own work between replays
        if inside == "acceptance":
            graph.replay()
            again = got[2]
        else:
            again = cache.accept(tokens, targets)
        assert same(cache, other) and again.n_path.tolist() == [0, 0, 0] and (again.path == -1).all() and again.next.tolist() == [-1] * 3
    assert int(cache.lens.max()) > 12                       # paths were kept
    with pytest.raises(ValueError, match="kept already"):
        other.accept(tokens, targets)
    pages_are_whole(cache)


def test_tables_that_do_not_fit_take_no_pages():
    pool = rg.Pool(400, 256, rg.LORA_F32, max_rank=1)
    with pytest.raises(torch.OutOfMemoryError):
        rg.KvDraftCache(pool, 40, LAYOUT, 65535, 1 << 21, 3, 7)      # a table of 22 TB
    assert pool.stats()["kv_pages"] == 0
    cache = rg.KvDraftCache(pool, LAYERS, LAYOUT, 3, 60, 90, 7)
    assert sorted(cache.stock.flatten().tolist()) == sorted(rg.lora_pool_kv_pages(pool.handle, 7))
