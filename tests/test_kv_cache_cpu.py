"""KvCache's bookkeeping and the order of what it does, on the host: a pool that only keeps its books, tables in
host memory, and streams that write down what is asked of them."""
import types

import pytest
import torch

import rank_gemm_unified_amd as rg

LAYOUT = rg.lora_kv_layout_t(4, 4, 64, 1)


class Stream:
    def __init__(self, name, handle, log):
        self.name, self.cuda_stream, self.log = name, handle, log

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))

    def synchronize(self):
        self.log.append((self.name, "is waited for"))


@pytest.fixture
def world(monkeypatch):
    """A cache of 2 layers and 3 rows over 40 pages, its log, and the streams `current`, `a` and `b`."""
    log = []
    w = types.SimpleNamespace(log=log, current=Stream("current", 0, log), a=Stream("a", 17, log), b=Stream("b", 18, log))
    by_handle = {s.cuda_stream: s for s in (w.current, w.a, w.b)}
    books = rg.Pool(40, 256, rg.LORA_BF16, max_rank=1, device=None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: by_handle[0])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: by_handle[handle])
    handle = lambda s: w.current.cuda_stream if s is None else s if isinstance(s, int) else s.cuda_stream

    def call(what):
        def run(*args, stream=None, **kw):
            log.append((by_handle[handle(stream)].name, what))
        return run

    def evict(layout, table, scores, lens, budget, first, last, in_place):
        log.append((w.current.name, "evicts"))
        n = torch.zeros_like(lens)
        n[: len(w.cache.rows)] = 1
        return table, scores, lens - n, table.clone(), n

    w.pool = types.SimpleNamespace(handle=books.handle, pages=torch.zeros(1), kv_write=call("writes"), kv_attend=call("attends"),
                                   kv_attend_chunk=call("attends"), kv_evict=evict, books=books,
                                   _where=lambda s: (handle(s), s is None))
    for name in ("grow", "drop", "free"):
        real = getattr(rg, f"lora_pool_{name}_kv")

        def logged(*args, real=real, name=name, **kw):
            if name != "grow":
                log.append(("pool", "takes back"))
            return real(*args, **kw)
        monkeypatch.setattr(rg, f"lora_pool_{name}_kv", logged)
    w.cache = rg.KvCache(w.pool, 2, LAYOUT, 3, 10, scores=True)
    return w


def _step(w, stream, counts={1: 2, 2: 1}):
    w.cache.append(counts)
    for layer in range(2):
        w.cache.write(layer, None, None, stream=stream)
        w.cache.attend(layer, None, stream=stream)
    w.log.clear()


@pytest.mark.parametrize("how", ["object", "handle"])
def test_append_comes_behind_the_streams_of_the_step(world, how):
    _step(world, world.a if how == "object" else 17)
    world.cache.append({1: 1})
    assert world.log[0] == ("current", "waits for", "a") and ("current", "is waited for") in world.log
    world.log.clear()
    world.cache.append({1: 1})                    # nothing ran in between
    assert not any(x[1] == "waits for" for x in world.log)


def test_steps_on_several_streams_and_on_the_current_one(world):
    _step(world, None)
    world.cache.append({1: 1})
    assert not any(x[1] == "waits for" for x in world.log)
    world.cache.write(0, None, None, stream=world.a)
    world.cache.attend(0, None, stream=world.b)
    world.cache.attend(1, None)
    world.log.clear()
    world.cache.append({1: 1})
    assert sorted(world.log[:2]) == [("current", "waits for", "a"), ("current", "waits for", "b")]


def test_a_step_on_what_was_then_the_current_stream(world):
    """The stream that was current at the step counts, not the one that is now."""
    was, world.current = world.current, world.b
    _step(world, None)
    world.current = was
    world.cache.append({1: 1})
    assert world.log[0] == ("current", "waits for", "b")


def test_eviction_comes_behind_the_step_and_pages_leave_after_it(world):
    _step(world, world.a)
    assert world.cache.evict(1) == {1: 1, 2: 1}
    assert world.log[:2] == [("current", "waits for", "a"), ("current", "evicts")]
    at = world.log.index(("pool", "takes back"))
    assert ("current", "is waited for") in world.log[2:at]


def test_finish_comes_behind_the_step(world):
    _step(world, world.a)
    world.cache.finish(1)
    assert ("current", "waits for", "a") in world.log
    assert world.cache.rows == {2: 1} and (world.cache.table[:, 0] == -1).all() and world.cache.lens.tolist() == [0, 1, 0]


def test_finish_gives_pages_back_when_nothing_reads_them(world):
    """Also with the step on the current stream: what takes the pages next may run on any."""
    for stream in (world.a, None):
        _step(world, stream)
        for rid in (1, 2):
            world.cache.finish(rid)
            at = world.log.index(("pool", "takes back"))
            assert ("current", "is waited for") in world.log[:at]
            world.log.clear()


def test_an_append_that_fails_leaves_the_free_list_as_it_was(world):
    """In its very order: the next pages handed out are the ones that would have been."""
    world.cache.append({1: 2, 2: 1})
    free = rg.lora_pool_free_list(world.pool.handle)
    held = {r: rg.lora_pool_kv_pages(world.pool.handle, r) for r in (1, 2)}
    with pytest.raises(rg.LoraError):
        world.cache.append({1: 3, 3: 3, 2: 2})
    assert rg.lora_pool_free_list(world.pool.handle) == free
    assert held == {r: rg.lora_pool_kv_pages(world.pool.handle, r) for r in (1, 2)}
    assert world.cache.rows == {1: 0, 2: 1} and rg.lora_pool_stats(world.pool.handle)["kv_requests"] == 2


def test_the_first_append_comes_behind_what_made_the_tables(world):
    """They are filled on the stream that was current then."""
    world.current = world.b
    world.cache.append({1: 2})
    assert world.log[0] == ("b", "waits for", "current")
