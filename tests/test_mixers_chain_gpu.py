"""The mixers as they are used: one decode step and one prompt of an attention layer and of a
recurrent layer, with the NVFP4 projections around them; the same captured in a graph and
replayed, on a side stream, and two batches on two streams at once."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import mixers as M

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, WIDTH = 8, 2, 128, 512


def _weights(rows, cols, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return nv.pack_weight(0.05 * torch.randn(rows, cols, device=DEV, generator=g))


class Layer:
    """An attention layer: fused q, k, v projection, append, attention, output projection."""

    def __init__(self, B, fp8, seed):
        g = torch.Generator(DEV).manual_seed(seed)
        self.B = B
        self.w_in, self.w_out = _weights((HEADS + 2 * KV) * DIM, WIDTH, seed), _weights(WIDTH, HEADS * DIM, seed + 1)
        amax = [torch.tensor([a], device=DEV) for a in (6.0, 6.0)] if fp8 else [None, None]
        self.cache = nv.PagedKVCache.empty(B * 20, 16, KV, DIM, DEV, *amax)
        self.cache.k.zero_(), self.cache.v.zero_()
        self.table = torch.randperm(B * 20, device=DEV, generator=g).int().view(B, 20)
        ang = torch.arange(320, device=DEV, dtype=torch.float64)[:, None] / 1e4 ** (
            torch.arange(0, 64, 2, device=DEV, dtype=torch.float64) / 64)
        self.rope = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.qkv = torch.empty(B, (HEADS + 2 * KV) * DIM, device=DEV)
        self.o = torch.empty(B, WIDTH, device=DEV)
        self.bufs = dict(q_out=torch.empty(B, HEADS, DIM, dtype=torch.bfloat16, device=DEV))
        self.attn = dict(out=torch.empty(B, HEADS, DIM, dtype=torch.bfloat16, device=DEV),
                         lse=torch.empty(B, HEADS, device=DEV), workspace=nv.Workspace(DEV))
        self.acts = [[torch.empty(B, k // 2, dtype=torch.uint8, device=DEV), torch.empty(B, k // 16, dtype=torch.uint8, device=DEV),
                      torch.empty(1, device=DEV)] for k in (WIDTH, HEADS * DIM)]
        self.ws = nv.Workspace(DEV)

    def slots(self):
        at = self.lens.long()
        return self.table.long().gather(1, (at // 16)[:, None])[:, 0] * 16 + at % 16

    def step(self, x):
        nv.linear(x, self.w_in, None, self.ws, out=self.qkv, act_out=self.acts[0])
        q, k, v = (p.view(self.B, -1, DIM) for p in self.qkv.split([HEADS * DIM, KV * DIM, KV * DIM], 1))
        q = nv.kv_append(k, v, self.cache, self.slots(), q=q, positions=self.lens.long(), rope=self.rope, **self.bufs)
        self.lens += 1
        out, _ = nv.attn_decode(q, self.cache, self.table, self.lens, max_len=320, **self.attn)
        nv.linear(out.view(self.B, -1), self.w_out, None, self.ws, out=self.o, act_out=self.acts[1])
        return self.o


def _oracle_attention(qkv_steps, rope, fp8, table, lens_end):
    """Attention of the last step from the fused projections of all steps, in 64 bits."""
    B = qkv_steps[0].shape[0]
    pages = table.size
    pool = [np.zeros((pages, 16, KV, DIM), np.uint8 if fp8 else np.uint16) for _ in range(2)]
    q_out = np.zeros((B, HEADS, DIM), np.uint16)
    for t, x in enumerate(qkv_steps):
        q, k, v = (p.reshape(B, -1, DIM) for p in np.split(x, [HEADS * DIM, (HEADS + KV) * DIM], 1))
        slots = table[:, t // 16].astype(np.int64) * 16 + t % 16
        M.append(q, k, v, rope, 64, False, np.full(B, t), slots, *pool, q_out, *((6.0, 6.0) if fp8 else (None, None)))
    val = [(M.kvfp8.decode_f32(p, 448.0).astype(np.float64) * (6.0 / 448)) if fp8 else M.bf16_value(p).astype(np.float64)
           for p in pool]
    return M.attend(M.bf16_value(q_out).astype(np.float64), *val, table, np.full(B, lens_end), 320, DIM ** -0.5, 0, KV)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_layer_decodes(fp8):
    """34 tokens through the layer: the cache and the last step's attention against the oracle."""
    say(f"[chain] attention layer fp8={fp8}")
    L = Layer(3, fp8, 1)
    g = torch.Generator(DEV).manual_seed(2)
    steps = []
    for _ in range(34):
        L.step(torch.randn(3, WIDTH, device=DEV, generator=g).bfloat16())
        steps.append(L.qkv.cpu().numpy())
    torch.cuda.synchronize()
    ref, _, mag, _ = _oracle_attention(steps, L.rope.cpu().numpy(), fp8, L.table.cpu().numpy(), 34)
    out = L.attn["out"].cpu().double().numpy()
    assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * mag + 1e-30).all()
    assert torch.isfinite(L.o).all()


def test_attention_layer_in_a_graph():
    """The decode step captured once and replayed; eager work and synchronizations between the
    replays; every replay equals the eager layer's step."""
    A, Bl = Layer(4, True, 5), Layer(4, True, 5)
    g = torch.Generator(DEV).manual_seed(6)
    xs = [torch.randn(4, WIDTH, device=DEV, generator=g).bfloat16() for _ in range(8)]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Bl.step(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    A.step(xs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Bl.step(x)
    for i in range(1, 8):
        x.copy_(xs[i])
        Bl.o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = A.step(xs[i])
        torch.cuda.synchronize()
        assert torch.equal(Bl.o, want), f"replay {i} differs"
        assert torch.equal(Bl.cache.k, A.cache.k) and torch.equal(Bl.lens, A.lens)


def test_long_attention_graphs_share_nothing_but_their_workspace():
    """Two captured calls over long sequences with one workspace, replayed in turn."""
    g = torch.Generator(DEV).manual_seed(7)
    cache = nv.PagedKVCache.empty(300, 64, 1, DIM, DEV)
    cache.k.normal_(generator=g), cache.v.normal_(generator=g)
    table = torch.randperm(300, device=DEV, generator=g).int()[:256].view(1, 256)
    ws = nv.Workspace(DEV)
    calls = []
    for n in (16000, 9000):
        q = torch.randn(1, 5, DIM, device=DEV, generator=g).bfloat16()
        lens = torch.tensor([n], dtype=torch.int32, device=DEV)
        out, lse = nv.attn_decode(q, cache, table, lens, workspace=ws)
        torch.cuda.synchronize()
        calls.append([q, lens, out.clone(), torch.empty_like(out), torch.empty_like(lse)])
    graphs = []
    for q, lens, _, out, lse in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            nv.attn_decode(q, cache, table, lens, workspace=ws, out=out, lse=lse)
    for i in range(6):
        c = calls[i % 2]
        c[3].fill_(float("nan"))
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        (torch.ones(8, device=DEV) * 2).sum().item()
        torch.cuda.synchronize()
        assert torch.equal(c[3], c[2]), f"replay {i}"


def _recurrent(T, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(*s, device=DEV, generator=g), dim=-1).bfloat16()  # noqa: E731
    return (unit(T, 2, DIM), unit(T, 2, DIM), torch.randn(T, 4, DIM, device=DEV, generator=g).bfloat16(),
            -torch.rand(T, 4, device=DEV, generator=g), torch.rand(T, 4, device=DEV, generator=g),
            torch.randn(3, 4, DIM, DIM, device=DEV, generator=g))


def test_recurrent_layer_in_a_graph():
    """A prompt and steps after it, captured together and replayed from the same states."""
    q, k, v, g, b, state = _recurrent(203, 3)
    ends = torch.tensor([0, 70, 200, 200], dtype=torch.int32, device=DEV)
    has = torch.tensor([1, 0, 1], dtype=torch.int32, device=DEV)
    start = state.clone()
    ws = nv.Workspace(DEV)
    out = torch.empty_like(v)

    def run():
        nv.gdn_prefill(q[:200], k[:200], v[:200], g[:200], b[:200], state, ends, has_state=has, workspace=ws, out=out[:200])
        nv.gdn_step(q[200:], k[200:], v[200:], g[200:], b[200:], state, out=out[200:])

    run()
    torch.cuda.synchronize()
    want, want_state = out.clone(), state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        state.copy_(start)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, want_state), f"replay {i}"


def test_side_streams_at_once():
    """Two batches on two streams, each with its own buffers, equal their runs alone."""
    sets = [_recurrent(300, s) for s in (21, 22)]
    ends = torch.tensor([0, 100, 300, 300], dtype=torch.int32, device=DEV)
    alone = []
    for q, k, v, g, b, state in sets:
        s = state.clone()
        alone.append((nv.gdn_prefill(q, k, v, g, b, s, ends), s))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for st, (q, k, v, g, b, state) in zip(streams, sets):
        got.append((nv.gdn_prefill(q, k, v, g, b, state, ends, stream=st), state))
    torch.cuda.synchronize()
    for (o, s), (p, t) in zip(got, alone):
        assert torch.equal(o, p) and torch.equal(s, t)
