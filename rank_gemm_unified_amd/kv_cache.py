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


class KvDraftCache:
    """The KV caches of up to max_seqs sequences whose steps are planned on the GPU: page tables, lengths and free pages live
    there, so that a step follows the one before without a word to the host, and can be captured into a graph whole.  For
    steps of drafted tokens (trees, of which the model keeps a path), single tokens (trees of one node) and prompts.

        cache = KvDraftCache(pool, layers, layout, max_seqs, max_tokens, groups, request, rope)
        cache.plan(counts, T)                         # new tokens of each sequence, T rows in all: a prompt
        q = cache.write(layer, q, k, v); o = cache.attend(layer, q)           # per layer, row by row as counts say
        cache.plan(counts, T, parents, max_nodes)     # a step of drafted trees: node 0 the token chosen last
        ... write, attend ...
        kept = cache.accept(tokens, targets)          # kept.path, n_path, next; the lengths are the kept tokens'
        cache.finish(rows)                            # their pages come back with the next plan

    counts: int32 [max_seqs] on the device, 0 for sequences that rest.  `groups` page groups (tokens_per_page tokens in all
    layers each) are taken from the pool under the id `request`, used in no other cache of it, and shared by the sequences;
    a sequence that they do not suffice for sits the step out (lora_kv_plan: its output is zero, its length stays; refused()
    says how many).  `lens`, `table`, `held`, `stock` and `state` are the same tensors throughout; `step` is the latest plan.

    Everything runs on the current stream and in its order; using the cache from another one is the caller's to order.  What a
    captured step reads and writes besides (rows, counts, parents, `step`) is its graph's: write(), attend() and accept() go with
    the plan() called last, captured or not, and may be called after each replay of a graph that holds it.

    Paths are kept once: accept() leaves the step without sequences (its step_lens go to 0), so that a second one, called or
    replayed, finds nothing (empty paths) and moves nothing.  Called again on a step whose plan() was not captured, it raises."""

    def __init__(self, pool, layers, layout, max_seqs, max_tokens, groups, request, rope=None):
        import rank_gemm_unified_amd as rg
        if pool.pages is None:
            raise ValueError("a bookkeeping-only pool holds no KV vectors")
        tpp = layout.tokens_per_page
        if not 1 <= max_tokens <= rg.LORA_MAX_KV_TOKENS - tpp:
            raise ValueError(f"max_tokens {max_tokens} not in [1, {rg.LORA_MAX_KV_TOKENS - tpp}]")
        if groups < 1 or max_seqs < 1:
            raise ValueError(f"{groups} page groups for {max_seqs} sequences")
        self._rg, self.pool, self.layers, self.layout, self.max_seqs = rg, pool, layers, layout, max_seqs
        self.max_tokens, self.request, self.rope, self._parents = max_tokens, request, rope, None
        i32 = dict(dtype=torch.int32, device=pool.pages.device)
        self.table = torch.full((layers, max_seqs, 2, -(-max_tokens // tpp)), -1, **i32)
        self.lens, self.held = torch.zeros(max_seqs, **i32), torch.zeros(max_seqs, **i32)
        self.state, self.stock = torch.tensor([0, groups, 0, 0], **i32), torch.empty((groups, layers, 2), **i32)
        ids = []                                           # (the pool's pages are taken when nothing else can be too much)
        try:
            for _ in range(groups):
                ids.append(rg.lora_pool_grow_kv(pool.handle, request, layers))
        except rg.LoraError:
            for group in reversed(ids):                    # the last taken first: the free list as it was
                rg.lora_pool_drop_kv(pool.handle, request, group[::-1])
            if ids:
                rg.lora_pool_free_kv(pool.handle, request)
            raise
        self.stock.copy_(torch.tensor(ids, dtype=torch.int32).view(groups, layers, 2))
        self.step = None

    def plan(self, counts, T, parents=None, max_nodes=None):
        """Plan a step of counts [max_seqs] new tokens, T rows at least (Pool.kv_plan).  parents: int32 [T], of trees of up to
        max_nodes nodes (None: 64); None: rows in a line, each seeing those before it."""
        max_nodes = 0 if parents is None else 64 if max_nodes is None else max_nodes
        words, new = (max_nodes + 63) // 64, lambda shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device=self.lens.device)
        step = self._rg.KvPlan(new(self.max_seqs), new(self.max_seqs + 1), new((self.layers, 2, T), torch.int64), new(T),
                               new((T, words), torch.int64) if words else None, self.lens, self.held, self.state)
        self.pool.kv_plan(self.layout, counts, self.lens, self.held, self.table, self.stock, self.state, T, self.max_tokens,
                          parents, max_nodes, out=step)
        self.step, self._parents, self._nodes, self._kept = step, parents, max_nodes, False
        self._captured = torch.cuda.is_current_stream_capturing()     # then its replays plan further steps, unseen

    def write(self, layer, q, k, v, q_out=None):
        """Layer `layer`'s rows of the step: K and V to their pages, and q, all turned by their positions if the cache has a
        Rope (Pool.kv_write_rope).  Returns the q to attend with: q_out, or, without a Rope, q itself."""
        if self.rope is None:
            self.pool.kv_write(self.layout, k, v, self.table[layer], self.step.step_lens, self.step.q_start)
            return q
        return self.pool.kv_write_rope(self.layout, self.rope, q, k, v, self.step.slots[layer], self.step.positions, q_out)

    def attend(self, layer, q, scale=None, max_len=None, out=None):
        """The step's attention in layer `layer` (Pool.kv_attend_tree, or kv_attend_chunk without parents).  max_len None: the
        longest a sequence may become."""
        max_len = self.max_tokens if max_len is None else max_len
        args = dict(scale=scale, max_len=max_len, out=out)
        if self._parents is None:
            return self.pool.kv_attend_chunk(self.layout, q, self.table[layer], self.step.step_lens, self.step.q_start, **args)
        return self.pool.kv_attend_tree(self.layout, q, self.table[layer], self.step.step_lens, self.step.q_start, self.step.mask,
                                        self._nodes, **args)

    def accept(self, tokens, targets):
        """Keep the path of each tree that the model agrees with (Pool.kv_accept): tokens, targets int32 [T], what each node
        stands for and what the model chose behind it.  Once a step."""
        if self._parents is None:
            raise ValueError("the step has no trees")
        if self._kept:
            raise ValueError("the step's paths are kept already")
        new, n = lambda *shape: torch.empty(shape, dtype=torch.int32, device=self.lens.device), self.max_seqs
        kept = self.pool.kv_accept(self.layout, self.table, self.step.step_lens, self.step.q_start, tokens, targets, self._parents,
                                   self._nodes, out=self._rg.KvAccepted(self.lens, new(n, self._nodes), new(n), new(n)))
        self.step.step_lens.zero_()
        self._kept = not (self._captured or torch.cuda.is_current_stream_capturing())
        return kept

    def finish(self, rows):
        """Sequences done: their rows are free, and the next plan takes their pages back.  A step that is planned already goes on
        without them: their output is zero from here on, and nothing of theirs is kept.  rows: a list, or an int64 tensor on the
        device, whose numbers outside [0, max_seqs) are no row."""
        n, rows = self.max_seqs, torch.as_tensor(rows, dtype=torch.int64)
        if not rows.is_cuda and rows.numel() and not 0 <= int(rows.min()) <= int(rows.max()) < n:
            raise ValueError(f"rows {rows.tolist()} not in [0, {n})")
        rows = rows.to(self.lens.device).reshape(-1)
        done = torch.zeros(n + 1, dtype=torch.bool, device=self.lens.device)     # (an index out of range would end the process)
        done = done.index_fill_(0, torch.where((rows >= 0) & (rows < n), rows, n), True)[:n]
        self.lens.masked_fill_(done, 0)
        if self.step is not None:
            self.step.step_lens.masked_fill_(done, 0)

    def refused(self):
        """Sequences that sat the latest step out although they had new tokens (waits for the device)."""
        return int(self.state[2])

    def close(self):
        """Every page back to the pool, when the device is done with them: whatever takes them next may write them on any
        stream."""
        torch.cuda.synchronize(self.lens.device)
        self._rg.lora_pool_free_kv(self.pool.handle, self.request)
