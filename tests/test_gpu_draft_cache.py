"""Steps of drafted tokens as a program runs them (KvDraftCache): a small model decodes with trees of drafts, some of them
right, and has to produce the tokens that it produces one by one in float64 on the host.

The argument: the device's logits are off by float32 rounding.  A sum has at most 256 terms whose sizes add up to 16 at the
most (normal weights over the root of the width, activations below 1), so that it is off by less than 256 * 2^-24 * 16 = 2.5e-4
if every rounding went the same way; every choice compared here has a lead of twice that."""
import numpy as np
import pytest
import torch

import rank_gemm_unified_amd as rg

pytestmark = pytest.mark.gpu

LAYERS, HEADS, KV, DIM, TPP, WIDTH, VOCAB = 2, 4, 2, 64, 3, 96, 40
LEAD = 5e-4


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Model:
    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        w = lambda *s: (rng.normal(size=s) / np.sqrt(s[0])).astype(np.float32)  # noqa: E731
        self.host = dict(e=rng.normal(size=(VOCAB, WIDTH)).astype(np.float32), u=w(WIDTH, VOCAB),
                         qkv=[w(WIDTH, (HEADS + 2 * KV) * DIM) for _ in range(LAYERS)], o=[w(HEADS * DIM, WIDTH) for _ in range(LAYERS)])
        up = lambda x: [torch.as_tensor(y, device="cuda") for y in x] if isinstance(x, list) else torch.as_tensor(x, device="cuda")  # noqa: E731
        self.dev = {k: up(v) for k, v in self.host.items()}
        self.rope = rg.Rope.of(256, DIM)
        self.turn = self.rope.table.double().cpu().numpy()

    def chosen(self, cache, tokens):
        """One pass over the step's rows: the token that the model chooses behind each."""
        x = self.dev["e"][tokens.long()]
        for layer in range(LAYERS):
            rows = x @ self.dev["qkv"][layer]
            q, k, v = rows[:, : HEADS * DIM], rows[:, HEADS * DIM: (HEADS + KV) * DIM], rows[:, (HEADS + KV) * DIM:]
            x = torch.tanh(x + cache.attend(layer, cache.write(layer, q, k, v)) @ self.dev["o"][layer])
        return (x @ self.dev["u"]).argmax(1).int()

    def next_token(self, tokens):
        """The token behind a whole sequence, in float64."""
        w = {k: [y.astype(np.float64) for y in v] if isinstance(v, list) else v.astype(np.float64) for k, v in self.host.items()}
        x, n = w["e"][tokens], len(tokens)

        def turned(y):
            y = y.reshape(n, -1, DIM)
            c, s = self.turn[:n, None, :, 0], self.turn[:n, None, :, 1]
            a, b = y[..., : DIM // 2], y[..., DIM // 2:]
            return np.concatenate([a * c - b * s, a * s + b * c], -1)

        for layer in range(LAYERS):
            rows = x @ w["qkv"][layer]
            q, k = turned(rows[:, : HEADS * DIM]), turned(rows[:, HEADS * DIM: (HEADS + KV) * DIM])
            v = rows[:, (HEADS + KV) * DIM:].reshape(n, KV, DIM)
            out = np.zeros((n, HEADS, DIM))
            for h in range(HEADS):
                z = np.where(np.tril(np.ones((n, n), bool)), q[:, h] @ k[:, h * KV // HEADS].T * DIM ** -0.5, -np.inf)
                p = np.exp(z - z.max(1, keepdims=True))
                out[:, h] = p / p.sum(1, keepdims=True) @ v[:, h * KV // HEADS]
            x = np.tanh(x + out.reshape(n, -1) @ w["o"][layer])
        z = np.sort((x[-1] @ w["u"])[:, None], 0)[:, 0]
        assert z[-1] - z[-2] > LEAD
        return int((x[-1] @ w["u"]).argmax())


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def setup(seed, lengths, new, groups=200, max_seqs=4, pages=1200):
    model, rng = Model(seed), np.random.default_rng(seed)
    pool = rg.Pool(pages, KV * DIM * TPP, rg.LORA_F32, max_rank=1)
    cache = rg.KvDraftCache(pool, LAYERS, rg.lora_kv_layout_t(HEADS, KV, DIM, TPP), max_seqs, 90, groups, 7, model.rope)
    prompts = [[int(t) for t in rng.integers(0, VOCAB, n)] for n in lengths]
    want = []
    for p in prompts:
        seq = list(p)
        for _ in range(new if p else 0):
            seq.append(model.next_token(seq))
        want.append(seq[len(p):])
    return model, pool, cache, rng, prompts, want


def drafts(rng, want, done, root, nodes):
    """A tree behind the token chosen last: a few of the right tokens, wrong ones beside and behind them."""
    tokens, parents, right = [root], [0], 0
    for i in range(1, nodes):
        if rng.random() < 0.5 and done + 1 < len(want):
            parents.append(right)
            tokens.append(want[done + 1])
            right, done = i, done + 1
        else:
            parents.append(int(rng.integers(0, i)))
            tokens.append(int(rng.integers(0, VOCAB)))
    return tokens, parents


def prompt(model, cache, prompts):
    counts = [len(p) for p in prompts]
    cache.plan(dev(counts), sum(counts) + 2)
    chosen = model.chosen(cache, dev([t for p in prompts for t in p] + [0, 0])).tolist()
    at = np.cumsum(counts) - 1
    return [chosen[a] if c else None for a, c in zip(at, counts)]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_drafted_tokens_are_the_model_s_own(seed, captured):
    model, pool, cache, rng, prompts, want = setup(seed, [5, 0, 11, 3], 24)
    roots, nodes = prompt(model, cache, prompts), 9
    got = [[] for _ in prompts]
    T = 3 * nodes + 4
    counts, tokens, parents = dev([0] * 4), dev([0] * T), dev([0] * T)
    kept = {}

    def step():
        cache.plan(counts, T, parents, nodes)
        kept["k"] = cache.accept(tokens, model.chosen(cache, tokens))

    graph = None
    if captured:
        side = torch.cuda.Stream()                          # a step without sequences, so that libraries are set up
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    most = 0
    for _ in range(40):
        live = [b for b, p in enumerate(prompts) if p and len(got[b]) < 20]
        if not live:
            break
        sizes, tok, par = [0] * 4, [], []
        for b in live:
            sizes[b] = int(rng.integers(1, nodes + 1))
            t, p = drafts(rng, want[b], len(got[b]), roots[b], sizes[b])
            tok, par = tok + t, par + p
        counts.copy_(dev(sizes))
        tokens.copy_(dev(tok + [0] * (T - len(tok))))
        parents.copy_(dev(par + [0] * (T - len(par))))
        if graph is None:
            step()
        else:
            graph.replay()
            torch.randn(100, device="cuda").sum().item()     # the program's own work between replays
        k, at = kept["k"], 0
        for b in range(4):
            if sizes[b]:
                path = k.path[b, : int(k.n_path[b])].tolist()
                got[b] += [tok[at + i] for i in path]
                roots[b] = int(k.next[b])
                most = max(most, len(path))
                assert int(cache.lens[b]) == len(prompts[b]) + len(got[b])
                at += sizes[b]
        assert cache.refused() == 0
    for b, p in enumerate(prompts):
        if p:
            assert got[b][:20] == want[b][:20], b
    assert most >= 3                                        # drafts were kept
    assert rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_OK
    # pages: what the lengths need is held, the rest is free, and none is lost or held twice
    cache.plan(dev([0] * 4), 1)
    held = [-(-int(n) // TPP) for n in cache.lens]
    assert cache.held.tolist() == held and int(cache.state[1]) == 200 - sum(held)
    head, free = cache.state.tolist()[:2]
    ids = [cache.stock[(head + i) % 200].flatten().tolist() for i in range(free)]
    ids += [cache.table[:, b, :, e].flatten().tolist() for b in range(4) for e in range(held[b])]
    flat = sorted(x for g in ids for x in g)
    assert flat == sorted(rg.lora_pool_kv_pages(pool.handle, 7))
    cache.close()
    assert pool.stats()["kv_pages"] == 0


def test_single_tokens_and_sequences_that_come_and_go():
    """Steps of one token each (trees of one node); a sequence ends and another takes its row and pages."""
    model, pool, cache, rng, prompts, want = setup(5, [4, 6], 10, groups=12, max_seqs=2)
    roots = prompt(model, cache, prompts)
    got, parents = [[], []], dev([0, 0])
    for _ in range(6):
        tokens = dev(roots)
        cache.plan(dev([1, 1]), 2, parents, 1)
        chosen = model.chosen(cache, tokens)
        with pytest.raises(ValueError, match="tokens"):
            cache.accept(tokens.long(), chosen)             # a refused call keeps nothing
        kept = cache.accept(tokens, chosen)
        with pytest.raises(ValueError, match="kept already"):
            cache.accept(tokens, tokens)
        for b in range(2):
            got[b].append(roots[b])
        roots = kept.next.tolist()
    assert got == [w[:6] for w in want]
    cache.finish([0])
    fresh = [int(t) for t in rng.integers(0, VOCAB, 9)]
    cache.plan(dev([9, 0]), 9)                              # nine tokens, three groups; four of twelve came back with this plan
    first = model.chosen(cache, dev(fresh)).tolist()[-1]
    assert cache.refused() == 0 and first == model.next_token(fresh)
    # more than there is: it sits the step out, its output is zero and nothing is written for it
    before, lens = pool.pages.clone(), cache.lens.tolist()
    cache.plan(dev([30, 0]), 30)
    assert cache.refused() == 1
    q = torch.randn((30, HEADS * DIM), device="cuda")
    kv = torch.randn((30, KV * DIM), device="cuda")
    out = cache.attend(0, cache.write(0, q, kv, kv, q_out=q))
    assert (out == 0).all() and torch.equal(pool.pages, before) and cache.lens.tolist() == lens
    with pytest.raises(ValueError, match="no trees"):
        cache.accept(dev([0] * 30), dev([0] * 30))
    assert rg.lora_check_device_errors(pool.handle, check=False) == rg.LORA_OK
    # without rotary embedding: the rows go in by the table
    plain = rg.KvDraftCache(pool, LAYERS, cache.layout, 2, 90, 4, 8)
    plain.plan(dev([2, 1]), 3)
    assert plain.write(1, q[:3], kv[:3], kv[:3]) is not None
    held = pool.pages[plain.table[1, 0, 0, 0].long(), : KV * DIM]
    assert torch.equal(held, kv[0])
    with pytest.raises(rg.LoraError):
        rg.KvDraftCache(pool, LAYERS, cache.layout, 2, 90, 10 ** 4, 9)
    assert pool.stats()["kv_requests"] == 2


def test_two_caches_on_two_streams():
    """Two caches over one pool, their steps queued on two streams at once."""
    model, pool, one, rng, prompts, want = setup(11, [5, 8], 8, groups=40, max_seqs=2)
    two = rg.KvDraftCache(pool, LAYERS, one.layout, 2, 90, 40, 8, model.rope)
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream(), torch.cuda.Stream()], []
    rows = dev([t for p in prompts for t in p])
    counts, steps = dev([5, 8]), dev([1, 1])
    parents = dev([0, 0])
    torch.cuda.synchronize()
    for cache, stream in zip((one, two), streams):
        with torch.cuda.stream(stream):
            cache.plan(counts, 13)
            root = model.chosen(cache, rows)[[4, 12]]
            seq = [root]
            for _ in range(6):
                cache.plan(steps, 2, parents, 1)
                root = cache.accept(root, model.chosen(cache, root)).next
                seq.append(root)
            out.append(torch.stack(seq, 1))
    torch.cuda.synchronize()
    assert out[0].tolist() == out[1].tolist() == [w[:7] for w in want]
