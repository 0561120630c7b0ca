"""Convenience owner of the KV caches of a batch of requests, in the layers of one model, over a pool:
the page tables, lengths and scores that the lora_kv_* calls take, kept in step with the pool's pages."""
from __future__ import annotations

import torch


class KvCache:
    """Up to max_seqs requests of up to max_tokens tokens each.  A request takes one row of every table;
    rows without a request have length 0 (padding).  A request's pages belong to one cache: its id is used in no other
    over the same pool.

        cache = KvCache(pool, layers, layout, max_seqs, max_tokens, scores=True)
        cache.append({7: 512, 9: 300})            # two prompts: pages, table rows, lengths
        cache.write(layer, k, v); o = cache.attend(layer, q)      # per layer, rows in cache row order
        cache.append({7: 1, 9: 1})                # a decode step
        cache.write(layer, k, v); o = cache.attend(layer, q)      # one row per cache row
        cache.evict(budget=256, keep_first=4, keep_last=64)       # pages go back to the pool
        cache.finish(7)

    append() decides what write() and attend() do next.  Where each row of the cache gets at most one
    token it is a decode step: k, v and q have max_seqs rows, row b for cache row b, and rows of requests
    that were not named are left alone (their output is zero).  Otherwise it is a chunk: the rows of the
    named requests one behind the other, in cache row order (`rows` of the request before that of a later
    one).  The device tensors (table, lens, step_lens, q_start, scores) are the same ones throughout, so a captured decode step
    may be replayed after each append().

    Streams: write() and attend() run on the stream they are given, or the current one.  append(), evict() and finish()
    change what those read: they put the current stream behind everything queued on the streams of the write() and
    attend() calls before, and return when their changes are in place, so the calls of the next step may run on any
    stream.  (A stream that was given has to live until then.)  Calls of one step on several streams are the caller's
    to order, and so is a graph replayed on another stream than the current one: the cache does not see it."""

    def __init__(self, pool, layers, layout, max_seqs, max_tokens, scores=False):
        import rank_gemm_unified_amd as rg
        self._rg, self.pool, self.layers, self.layout, self.max_seqs = rg, pool, layers, layout, max_seqs
        self.tpp = layout.tokens_per_page
        self.max_pages = -(-max_tokens // self.tpp)
        dev = None if pool.pages is None else pool.pages.device
        if dev is None:
            raise ValueError("a bookkeeping-only pool holds no KV vectors")
        if not 1 <= max_tokens <= rg.LORA_MAX_KV_TOKENS - self.tpp:
            raise ValueError(f"max_tokens {max_tokens} not in [1, {rg.LORA_MAX_KV_TOKENS - self.tpp}]")
        self.max_tokens = max_tokens
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((layers, max_seqs, 2, self.max_pages), -1, **i32)
        self.lens = torch.zeros(max_seqs, **i32)          # every request's tokens
        self.step_lens = torch.zeros(max_seqs, **i32)     # of the requests of this step, 0 for the others
        self.q_start = torch.zeros(max_seqs + 1, **i32)
        self.scores = torch.zeros((layers, max_seqs, self.max_pages * self.tpp), dtype=torch.float32,
                                  device=dev) if scores else None
        self.rows = {}                                    # request -> row
        self.length = [0] * max_seqs
        self._chunk = False
        self._used = {}                                   # handle -> stream that calls of this step ran on
        self._runs_on(None)                               # what filled the tensors above

    def _runs_on(self, stream):
        """Note the stream of a call: what changes the cache next comes behind it."""
        handle = self.pool._where(stream)[0]
        if handle not in self._used:
            dev = self.table.device
            if stream is None:
                stream = torch.cuda.current_stream(dev)
            elif isinstance(stream, int):
                stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
            self._used[handle] = stream

    def _behind_the_step(self):
        """Put the current stream behind the calls since the last change; returns it."""
        now = torch.cuda.current_stream(self.table.device)
        for handle, stream in self._used.items():
            if handle != now.cuda_stream:
                now.wait_stream(stream)
        self._used = {now.cuda_stream: now}
        return now

    def _in_place(self, now):
        """Wait until the changes, and so the calls they came behind, are done."""
        now.synchronize()
        self._used = {}

    def _pages(self, tokens):
        return -(-tokens // self.tpp)

    def append(self, counts):
        """counts: {request id: new tokens (>= 1)}; a request that is new takes a free row.  Takes the pages
        from the pool and writes them into the tables; nothing is changed if the pool has too few
        (LoraError, enomem), a request would outgrow max_tokens or no row is free (ValueError)."""
        rows, fresh = dict(self.rows), []
        for rid, n in counts.items():
            if n < 1:
                raise ValueError(f"request {rid}: {n} new tokens")
            if rid not in rows:
                free = [r for r in range(self.max_seqs) if r not in rows.values()]
                if not free:
                    raise ValueError(f"no free row for request {rid}: {self.max_seqs} are in use")
                rows[rid] = free[0]
                fresh.append(rid)
            if self.length[rows[rid]] + n > self.max_tokens:
                raise ValueError(f"request {rid}: {self.length[rows[rid]]} + {n} tokens, {self.max_tokens} at most")
        got, entries = {}, []
        try:
            for rid, n in counts.items():
                row = rows[rid]
                for e in range(self._pages(self.length[row]), self._pages(self.length[row] + n)):
                    ids = self._rg.lora_pool_grow_kv(self.pool.handle, rid, self.layers)
                    got.setdefault(rid, []).extend(ids)
                    entries.append((row, e, ids))
        except self._rg.LoraError:
            for rid, ids in reversed(got.items()):          # the last taken first: the free list as it was
                self._rg.lora_pool_drop_kv(self.pool.handle, rid, ids[::-1])
                if rid in fresh:
                    self._rg.lora_pool_free_kv(self.pool.handle, rid)
            raise
        self.rows = rows
        now = self._behind_the_step()
        if entries:
            dev = self.table.device
            at = torch.tensor([(r, e) for r, e, _ in entries], device=dev)
            ids = torch.tensor([i for _, _, i in entries], dtype=torch.int32, device=dev).view(-1, self.layers, 2)
            self.table[:, at[:, 0], :, at[:, 1]] = ids
        new = [0] * self.max_seqs
        for rid, n in counts.items():
            new[rows[rid]] = n
            self.length[rows[rid]] += n
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self._chunk = max(new) > 1
        self.lens.copy_(torch.tensor(self.length, dtype=torch.int32))
        self.step_lens.copy_(torch.tensor([l if n else 0 for l, n in zip(self.length, new)], dtype=torch.int32))
        self.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
        self._in_place(now)

    def write(self, layer, k, v, stream=None):
        """The step's K and V rows into layer `layer`'s pages (Pool.kv_write)."""
        self._runs_on(stream)
        self.pool.kv_write(self.layout, k, v, self.table[layer], self.step_lens, self.q_start if self._chunk else None,
                           stream=stream)

    def attend(self, layer, q, scale=None, max_len=None, out=None, stream=None):
        """The step's attention in layer `layer` (Pool.kv_attend or kv_attend_chunk), its weights added to the
        layer's scores if the cache keeps them.  max_len None: the longest a request may become."""
        self._runs_on(stream)
        sc = None if self.scores is None else self.scores[layer]
        args = dict(scale=scale, max_len=self.max_tokens if max_len is None else max_len, out=out, scores=sc, prior=sc,
                    stream=stream)
        if self._chunk:
            return self.pool.kv_attend_chunk(self.layout, q, self.table[layer], self.step_lens, self.q_start, **args)
        return self.pool.kv_attend(self.layout, q, self.table[layer], self.step_lens, **args)

    def evict(self, budget, keep_first=0, keep_last=0):
        """Thin every request out to about `budget` tokens (Pool.kv_evict) and give its pages back to the pool,
        when the step's calls are done with them.  Returns {request: tokens that left}."""
        if self.scores is None:
            raise ValueError("this cache keeps no scores")
        now = self._behind_the_step()
        *_, lens, dropped, n = self.pool.kv_evict(self.layout, self.table, self.scores, self.lens, budget, keep_first,
                                                  keep_last, in_place=True)
        self.lens.copy_(lens)
        self.step_lens.zero_()                            # the next step begins with append()
        n, gone = n.tolist(), {}
        most = max(n, default=0)
        ids = dropped[..., :most].cpu() if most else None
        self._in_place(now)
        for rid, row in self.rows.items():
            if n[row]:
                self._rg.lora_pool_drop_kv(self.pool.handle, rid, ids[:, row, :, : n[row]].reshape(-1).numpy())
                self.length[row] -= n[row] * self.tpp
                gone[rid] = n[row] * self.tpp
        return gone

    def finish(self, rid):
        """Request done: its row is free, and its pages go back to the pool, once the step's calls, which may read them,
        are done: whatever takes the pages next may write them on any stream."""
        row = self.rows.pop(rid)
        self.length[row] = 0
        now = self._behind_the_step()
        self.table[:, row] = -1
        self.lens[row] = 0
        self.step_lens[row] = 0
        if self.scores is not None:
            self.scores[:, row] = 0
        self._in_place(now)
        self._rg.lora_pool_free_kv(self.pool.handle, rid)
