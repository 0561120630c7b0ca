"""KvCache with its calls on a stream of their own, against the same steps one after the other."""
import pytest
import torch

import rank_gemm_unified_amd as rg
from test_gpu_kv import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

NH, NKV, DIM, H, LAYERS, ROWS, MOST = 8, 2, 64, 256, 2, 3, 700


class Twin:
    """Two caches over pools of the same content that make the same steps: `serial` on the current stream, waited for
    after each; `aside` on a stream of its own that is kept busy, not waited for."""

    def __init__(self, dtype=torch.bfloat16):
        self.layout, self.dt = rg.lora_kv_layout_t(NH, NKV, DIM, 2), dtype
        code = rg.LORA_BF16 if dtype is torch.bfloat16 else rg.LORA_F32
        self.pools = [rg.Pool(2 * LAYERS * ROWS * 360, H, code, max_rank=1) for _ in range(2)]
        for p in self.pools:
            p.pages.zero_()
        self.caches = [rg.KvCache(p, LAYERS, self.layout, ROWS, MOST, scores=True) for p in self.pools]
        self.stream = torch.cuda.Stream()
        self.g = torch.Generator(device="cuda").manual_seed(31)
        self.busy = torch.randn((4096, 4096), device="cuda").bfloat16()
        self.outs = [[], []]
        torch.cuda.synchronize()

    def step(self, counts):
        T = sum(counts.values()) if max(counts.values()) > 1 else ROWS
        rows = [[torch.empty((T, w * DIM), dtype=self.dt, device="cuda").normal_(generator=self.g) for w in (NKV, NKV, NH)]
                for _ in range(LAYERS)]
        serial, aside = self.caches
        serial.append(counts)
        for layer, (k, v, q) in enumerate(rows):
            serial.write(layer, k, v)
            self.outs[0].append(serial.attend(layer, q))
        torch.cuda.synchronize()
        aside.append(counts)
        with torch.cuda.stream(self.stream):                 # a few milliseconds of work before the step's
            for _ in range(24):
                torch.mm(self.busy, self.busy)
        for layer, (k, v, q) in enumerate(rows):
            aside.write(layer, k, v, stream=self.stream)
            self.outs[1].append(aside.attend(layer, q, stream=self.stream if layer else self.stream.cuda_stream))
        self.rows = rows                                     # read until the next step at least

    def same_outputs(self):
        torch.cuda.synchronize()
        assert len(self.outs[0]) == len(self.outs[1])
        for i, (x, y) in enumerate(zip(*self.outs)):
            assert torch.equal(x, y), i

    def same(self):
        self.same_outputs()
        a, b = self.caches
        assert a.length == b.length and a.rows == b.rows
        for name in ("table", "lens", "step_lens", "q_start", "scores"):
            x, y = getattr(a, name), getattr(b, name)
            assert torch.equal(x, y), name
        assert torch.equal(self.pools[0].pages, self.pools[1].pages)
        assert rg.lora_pool_free_list(self.pools[0].handle) == rg.lora_pool_free_list(self.pools[1].handle)
        for p in self.pools:
            assert rg.lora_check_device_errors(p.handle, check=False) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_on_another_stream(dtype):
    """append, evict and finish come behind the step before them, wherever it runs."""
    t = Twin(dtype)
    t.step({1: 300, 2: 41})
    t.step({1: 1, 2: 1})
    t.step({1: 1, 3: 1})                                      # row 1 pauses: its lengths of the step before change
    gone = [c.evict(100, 4, 20) for c in t.caches]
    assert gone[0] == gone[1] and gone[0]
    t.same()
    t.step({2: 1, 3: 1})
    for c in t.caches:
        c.finish(2)
    t.step({3: 200, 4: 50})
    t.step({1: 1, 3: 1, 4: 1})
    for rid in (1, 3, 4):
        for c in t.caches:
            c.finish(rid)
    t.same()


def test_steps_under_another_current_stream():
    """The streams that were current at the calls count."""
    t = Twin()
    t.step({1: 100, 2: 33})
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        for c in t.caches:
            assert c.evict(50, 2, 2)
    t.same()
    with torch.cuda.stream(other):
        t.step({1: 1, 2: 1})
    for c in t.caches:
        c.finish(1)
    t.step({2: 1, 5: 1})
    t.same()


def test_pages_of_a_finished_request_may_be_written_at_once():
    """What takes them next, an adapter loaded on a stream of its own, say, changes nothing that the step reads."""
    t = Twin()
    t.step({1: 400, 2: 300})
    for c, p in zip(t.caches, t.pools):
        pages = [rg.lora_pool_kv_pages(p.handle, r) for r in (1, 2)]
        c.finish(1)
        c.finish(2)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            p.pages[torch.as_tensor(sum(pages, [])).to("cuda", non_blocking=False)] = float("nan")
        s.synchronize()
    t.same_outputs()


def test_a_captured_step_replayed_after_each_append():
    """write and attend of a decode step, captured once and replayed, against the same steps run eagerly."""
    t = Twin()
    t.step({1: 300, 2: 41})
    torch.cuda.synchronize()
    eager, replayed = t.caches
    k, v, q = (torch.zeros((LAYERS, ROWS, w * DIM), dtype=t.dt, device="cuda") for w in (NKV, NKV, NH))

    def calls(cache):
        outs = []
        for layer in range(LAYERS):
            cache.write(layer, k[layer], v[layer])
            outs.append(cache.attend(layer, q[layer]))
        return outs

    graph = None
    for counts in ({1: 1, 2: 1}, {1: 1}, {2: 1, 3: 1}, {1: 1, 2: 1, 3: 1}):
        for x in (k, v, q):
            x.normal_(generator=t.g)
        eager.append(counts)
        want = calls(eager)
        replayed.append(counts)
        if graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = calls(replayed)
        for o in outs:
            o.fill_(7.25)
        graph.replay()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), counts
        if counts == {1: 1}:
            assert [c.evict(200, 2, 9) for c in t.caches] == [{1: 102}] * 2
    t.same()
    for rid in (1, 2, 3):
        for c in t.caches:
            c.finish(rid)
    t.same()
