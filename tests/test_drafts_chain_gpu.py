"""The operators for drafted tokens as they are used together: greedy decoding of a small model with
drafted trees against the same model token by token, the step captured in a graph and replayed, on a side
stream, and two batches on two streams at once."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, WIDTH, VOCAB, PAGE, PAGES, LAYERS = 8, 2, 128, 512, 1000, 16, 24, 2


class Model:
    """Two attention layers between projections, and an output projection to logits.  The projections are
    NVFP4's with calibrated activation scales, or binary64 products, whose rows do not depend on the rows beside
    them (of an NVFP4 product they do, in the last bits of its sums, and the next activation's 4 bits turn
    such a bit into a step now and then)."""

    def __init__(self, B, fp8, seed, nvfp4):
        g = torch.Generator(DEV).manual_seed(seed)
        self.nvfp4, self.keep = nvfp4, False
        w = lambda n, k, s: (nv.pack_weight if nvfp4 else torch.Tensor.double)(s * torch.randn(n, k, device=DEV, generator=g))  # noqa: E731
        self.B, self.embed = B, torch.randn(VOCAB, WIDTH, device=DEV, generator=g)
        self.w_in = [w((HEADS + 2 * KV) * DIM, WIDTH, 0.06) for _ in range(LAYERS)]
        self.w_out = [w(WIDTH, HEADS * DIM, 0.06) for _ in range(LAYERS)]
        self.w_logits = w(VOCAB, WIDTH, 0.1)
        self.norms = [[1 + 0.1 * torch.randn(DIM, device=DEV, generator=g) for _ in range(2)] for _ in range(LAYERS)]
        self.amax = torch.tensor([8.0], device=DEV)
        ang = torch.arange(512, device=DEV, dtype=torch.float64)[:, None] / 1e4 ** (
            torch.arange(0, DIM, 2, device=DEV, dtype=torch.float64) / DIM)
        self.rope = torch.cat([ang.cos(), ang.sin()], 1).float()
        calibrated = [torch.tensor([a], device=DEV) for a in (6.0, 12.0)] if fp8 else [None, None]
        self.caches = [nv.PagedKVCache.empty(B * PAGES, PAGE, KV, DIM, DEV, *calibrated) for _ in range(LAYERS)]
        for c in self.caches:
            c.k.zero_(), c.v.zero_()
        self.table = torch.randperm(B * PAGES, device=DEV, generator=g).int().view(B, PAGES)
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.ws, self.linear_ws = nv.Workspace(DEV), nv.Workspace(DEV)

    def slots(self, at):
        return self.table.long().gather(1, at // PAGE) * PAGE + at % PAGE

    def linear(self, x, w):
        return nv.linear(x.bfloat16(), w, self.amax, self.linear_ws)[0] if self.nvfp4 else (x.double() @ w.T).float()

    def layer(self, i, x, at, depth, attend):
        """Tokens x [B, W, WIDTH] at cache rows lens + at and positions lens + depth through layer i."""
        B, W = x.shape[:2]
        rows = self.linear(x.view(B * W, WIDTH), self.w_in[i])
        q, k, v = (p.view(B * W, -1, DIM) for p in rows.split([HEADS * DIM, KV * DIM, KV * DIM], 1))
        base = self.lens.long()[:, None]
        q = nv.kv_append(k, v, self.caches[i], self.slots(base + at).flatten(), q=q, positions=(base + depth).flatten(),
                         rope=self.rope, q_norm=self.norms[i][0], k_norm=self.norms[i][1])
        o = attend(q.view(B, W, HEADS, DIM), self.caches[i])
        y = self.linear(o.reshape(B * W, HEADS * DIM), self.w_out[i])
        return x + y.view(B, W, WIDTH)

    def logits(self, tokens, at, depth, attend):
        x = self.embed[tokens]
        for i in range(LAYERS):
            x = self.layer(i, x, at, depth, attend)
        x = torch.nn.functional.rms_norm(x, (WIDTH,))
        return self.linear(x.flatten(0, 1), self.w_logits).view(*tokens.shape, VOCAB)

    def token(self, tokens):
        """One new token a sequence [B, 1] -> logits [B, 1, VOCAB]."""
        zero = torch.zeros(1, 1, dtype=torch.int64, device=DEV)

        def attend(q, cache):
            out, _ = nv.attn_decode(q[:, 0], cache, self.table, self.lens + 1, max_len=PAGES * PAGE, workspace=self.ws)
            return out
        out = self.logits(tokens, zero, zero, attend)
        self.lens += 1
        return out

    def tree(self, tokens, parents, depth, **verify):
        """A tree of drafted tokens [B, W]: what the model makes of it, with the caches and lengths moved on."""
        at = torch.arange(tokens.shape[1], device=DEV)[None]

        def attend(q, cache):
            out, _ = nv.attn_tree(q, cache, self.table, self.lens, parents, max_len=PAGES * PAGE - tokens.shape[1], workspace=self.ws)
            return out
        logits = self.logits(tokens, at, depth, attend)
        said, path, counts = nv.verify_drafts(logits, tokens, parents, workspace=self.ws, **verify)
        self.before = [(c.k.clone(), c.v.clone()) for c in self.caches] if self.keep else None
        nv.kv_compact(self.table, self.lens, path, counts, self.caches)
        self.lens += counts
        return logits, said, path, counts


def _tree(B):
    """The root, two children, three grandchildren, two below them, one padded node."""
    parents = [-1, 0, 0, 1, 1, 2, 3, 5, -2]
    depth = [0, 1, 1, 2, 2, 2, 3, 3, 0]
    return (torch.tensor([parents] * B, dtype=torch.int32, device=DEV), torch.tensor([depth] * B, device=DEV))


def _greedy(fp8, seed, steps):
    """Tokens of greedy decoding, token by token."""
    m = Model(3, fp8, seed, False)
    t = torch.tensor([[5], [77], [901]], device=DEV)
    tokens = [t]
    for _ in range(steps):
        t = m.token(t).argmax(-1)
        tokens.append(t)
    return torch.cat(tokens, 1)


def test_drafted_trees_give_the_tokens_of_greedy_decoding():
    """Over a bf16 cache.  (Tree and single tokens sum in other orders, so that a layer's input differs in its last
    bits now and then; a code of an E4M3 cache makes a sixteenth of that, which moves logits by up to 0.04, and
    some of 180 tokens have two logits that are closer: there equal tokens are no test.)"""
    fp8, steps, seed = False, 60, 11
    say("[drafts] greedy decoding with trees")
    want = _greedy(fp8, seed, steps)
    m = Model(3, fp8, seed, False)
    m.keep = True
    parents, depth = _tree(3)
    r = np.random.default_rng(3)
    last = want[:, :1].clone()
    done, calls, gained = [0, 0, 0], 0, 0
    while min(done) < steps - 9:
        # drafts: the right continuation down one branch, here and there with a wrong token in it
        drafts = torch.from_numpy(r.integers(0, VOCAB, (3, 9))).to(DEV)
        drafts[:, 0] = last[:, 0]
        for b in range(3):
            branch = [2, 5, 7] if r.random() < 0.5 else [1, int(r.choice([3, 4])), 6]
            for d, node in enumerate(branch):
                if r.random() < 0.8 and done[b] + 1 + d <= steps:
                    drafts[b, node] = want[b, done[b] + 1 + d]
        logits, said, path, counts = m.tree(drafts, parents, depth)
        for b in range(3):
            n = int(counts[b])
            assert said[b, :n].tolist() == want[b, done[b] + 1: done[b] + 1 + n].tolist(), (b, done[b])
            # the rows of the path lie where the sequence goes on, bit for bit
            at = torch.arange(n, device=DEV) + done[b]
            src, dst = (m.table[b].long()[x // PAGE] * PAGE + x % PAGE for x in (done[b] + path[b, :n].long(), at))
            for old, c in zip(m.before, m.caches):
                for x, y in zip(old, (c.k, c.v)):
                    bits = (lambda t: t.view(torch.uint8).flatten(0, 1).flatten(1))
                    assert torch.equal(bits(x)[src], bits(y)[dst])
            done[b] += n
            gained += n - 1
        calls += 1
        last = said.gather(1, (counts.long() - 1)[:, None])
        assert m.lens.tolist() == done
    assert gained > calls                                  # more than one draft a call was accepted


def _step(m, tokens, parents, depth, uniforms, temperature):
    return m.tree(tokens, parents, depth, temperature=temperature, uniforms=uniforms)


def test_a_captured_step_replays():
    """One step with drawn tokens captured once and replayed, eager work and synchronizations between the replays:
    every replay equals the eager model's step, caches and lengths among it."""
    say("[drafts] a step in a graph")
    A, C = Model(2, True, 21, True), Model(2, True, 21, True)
    parents, depth = _tree(2)
    g = torch.Generator(DEV).manual_seed(4)
    feeds = [(torch.randint(0, VOCAB, (2, 9), device=DEV, generator=g), torch.rand(2, 10, device=DEV, generator=g)) for _ in range(6)]
    heat = torch.tensor([0.7, 1.1], device=DEV)
    tokens, uniforms = feeds[0][0].clone(), feeds[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(C, tokens, parents, depth, uniforms, heat)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    _step(A, *feeds[0][:1], parents, depth, feeds[0][1], heat)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(C, tokens, parents, depth, uniforms, heat)
    for i in range(1, 6):
        tokens.copy_(feeds[i][0]), uniforms.copy_(feeds[i][1])
        got[1].fill_(-9)
        torch.cuda.synchronize()
        graph.replay()
        (torch.ones(8, device=DEV) * 2).sum().item()
        torch.cuda.synchronize()
        want = _step(A, feeds[i][0], parents, depth, feeds[i][1], heat)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), f"replay {i}"
        assert torch.equal(A.lens, C.lens)
        for x, y in zip(A.caches, C.caches):
            assert torch.equal(x.k, y.k) and torch.equal(x.v, y.v)


def test_two_streams_and_the_stream_argument():
    say("[drafts] two streams")
    g = torch.Generator(DEV).manual_seed(6)
    cache = nv.PagedKVCache.empty(80, PAGE, KV, DIM, DEV)
    cache.k.normal_(generator=g), cache.v.normal_(generator=g)
    table = torch.randperm(80, device=DEV, generator=g).int().view(2, 40)
    lens = torch.tensor([600, 333], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 9, HEADS, DIM, device=DEV, generator=g).bfloat16()
    parents, _ = _tree(2)
    logits, other = (3 * torch.randn(2, 9, 20000, device=DEV, generator=g) for _ in range(2))
    drafts, u = torch.randint(0, 20000, (2, 9), device=DEV, generator=g), torch.rand(2, 10, device=DEV, generator=g)
    heat = torch.ones(2, device=DEV)
    want = nv.attn_tree(q, cache, table, lens, parents)
    said = [nv.verify_drafts(logits, drafts, parents, heat, u), nv.verify_drafts(logits, drafts, None, heat, u, draft_logits=other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [nv.Workspace(DEV) for _ in range(2)]
    for _ in range(5):
        outs = []
        for s, ws in zip(streams, spaces):
            outs.append(nv.attn_tree(q, cache, table, lens, parents, workspace=ws, stream=s))
            outs.append(nv.verify_drafts(logits, drafts, parents, heat, u, workspace=ws, stream=s))
            outs.append(nv.verify_drafts(logits, drafts, None, heat, u, draft_logits=other, workspace=ws, stream=s))
        torch.cuda.synchronize()
        for got, ref in zip(outs, [want, *said] * 2):
            for x, y in zip(got, ref):
                assert torch.equal(x, y)
    copies = [nv.PagedKVCache(cache.k.clone(), cache.v.clone()) for _ in range(2)]
    torch.cuda.synchronize()
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    path, counts, src, dst = i(0, 2, 5, -1, 0, 1, 4, -1).view(2, 4), i(3, 3), i(3, 9), i(60, 61)
    torch.cuda.synchronize()
    for c, s in zip(copies, (None, streams[0])):
        nv.kv_compact(table, lens, path, counts, c, stream=s)
        nv.kv_copy_pages(src, dst, c, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(copies[0].k, copies[1].k) and torch.equal(copies[0].v, copies[1].v)
    assert not torch.equal(copies[0].k, cache.k)


def test_forked_sequences_go_on_apart():
    """Two answers to one prompt: full pages shared in the block tables, the last one copied; what one of them
    appends and attends to leaves the other as it was."""
    say("[drafts] a fork")
    g = torch.Generator(DEV).manual_seed(8)
    cache = nv.PagedKVCache.empty(12, PAGE, KV, DIM, DEV)
    rows = lambda n, h: torch.randn(n, h, DIM, device=DEV, generator=g).bfloat16()  # noqa: E731
    n = 3 * PAGE + 5
    nv.kv_append(rows(n, KV), rows(n, KV), cache, torch.arange(n, device=DEV))
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    nv.kv_copy_pages(i(3), i(9), cache)
    table = i(0, 1, 2, 3, 0, 1, 2, 9).view(2, 4)
    k, v, q = rows(4, KV), rows(4, KV), rows(4, HEADS).view(2, 2, HEADS, DIM)
    slots = torch.tensor([3 * PAGE + 5, 3 * PAGE + 6, 9 * PAGE + 5, 9 * PAGE + 6], device=DEV)
    nv.kv_append(k, v, cache, slots)
    both, _ = nv.attn_tree(q, cache, table, i(n, n))
    alone = nv.PagedKVCache.empty(12, PAGE, KV, DIM, DEV)
    for b in range(2):
        alone.k.copy_(cache.k), alone.v.copy_(cache.v)
        alone.k[9 if b == 0 else 3] = float("nan")
        one, _ = nv.attn_tree(q[b:b + 1], alone, table[b:b + 1], i(n))
        torch.cuda.synchronize()
        assert torch.equal(one[0], both[b]) and torch.isfinite(one.float()).all()
    assert not torch.equal(both[0], both[1])
