"""More of the mixers as they are used: a recurrent layer between its NVFP4 projections, the calls
by name, and a cache beyond the 2^31st element."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import mixers as M

pytestmark = pytest.mark.gpu
HK, HV, D, WIDTH = 2, 4, 128, 512
QKV = (2 * HK + HV) * D


class Recurrent:
    """A recurrent layer: one fused projection to q, k, v, beta and alpha, the gates and unit
    queries and keys as the model makes them, the delta rule, and the output projection.  The
    projections give fp32 rows; the mixers of this layer take bf16."""

    def __init__(self, seed):
        g = torch.Generator(DEV).manual_seed(seed)
        cols = [HK * D, HK * D, HV * D, HV, HV]
        ends = np.cumsum(cols)
        w = 0.05 * torch.randn(int(ends[-1]), WIDTH, device=DEV, generator=g)
        self.w_in = nv.pack_weight(w, [(int(e - n), int(e)) for n, e in zip(cols, ends)])
        self.w_out = nv.pack_weight(0.05 * torch.randn(WIDTH, HV * D, device=DEV, generator=g))
        self.rate = 1 + 3 * torch.rand(HV, device=DEV, generator=g)

    def split(self, rows):
        """The mixer's inputs from the fused rows."""
        q, k, v, b, a = rows.split([HK * D, HK * D, HV * D, HV, HV], 1)
        unit = lambda x: torch.nn.functional.normalize(x.reshape(-1, HK, D), dim=-1).bfloat16()  # noqa: E731
        return (unit(q), unit(k), v.reshape(-1, HV, D).bfloat16(), -self.rate * torch.nn.functional.softplus(a), torch.sigmoid(b))

    def project(self, x):
        out, _ = nv.linear(x, self.w_in)
        return self.split(out)

    def out(self, o):
        y, _ = nv.linear(o.reshape(-1, HV * D), self.w_out)
        return y


def _f64(t):
    return t.detach().cpu().double().numpy()


def _check(parts, ends, has, start, out, state, index):
    """Against the recurrence in 64 bits, with the bounds of test_gdn_gpu.py."""
    q, k, v, g, b = (_f64(p) for p in parts)
    ref, S, L = M.gdn(q, k, v, g, b, _f64(start), index, ends, has, D ** -0.5)
    out, state = _f64(out), _f64(state)
    for s in range(len(ends) - 1):
        r, n = slice(ends[s], ends[s + 1]), ends[s + 1] - ends[s]
        for h in range(HV):
            big = L[index[s], h] + (np.linalg.norm(v[r, h], axis=-1).max() if n else 0)
            tol = 8 * np.sqrt(n + 8) * 2.0 ** -24 * big
            assert np.linalg.norm(state[index[s], h] - S[index[s], h]) <= tol
            qn = np.linalg.norm(q[r, h // (HV // HK)], axis=-1, keepdims=True)
            d = np.abs(out[r, h] - ref[r, h])
            assert (d <= 2.0 ** -8 * np.abs(ref[r, h]) + D ** -0.5 * qn * (tol + 2.0 ** -14 * big) + 1e-30).all()


def test_recurrent_layer_between_its_projections():
    """Two prompts, then six tokens each, through linear -> gdn -> linear; the same in a graph."""
    say("[layers] linear -> gdn_prefill -> linear, linear -> gdn_step -> linear")
    layer = Recurrent(1)
    g = torch.Generator(DEV).manual_seed(2)
    lens, steps = [70, 133], 6
    x = torch.randn(sum(lens), WIDTH, device=DEV, generator=g).bfloat16()
    xs = [torch.randn(2, WIDTH, device=DEV, generator=g).bfloat16() for _ in range(steps)]
    ends = np.array([0, 70, 203])
    cu, index = torch.tensor(ends, dtype=torch.int32, device=DEV), torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    state = torch.randn(3, HV, D, D, device=DEV, generator=g)
    start = state.clone()

    parts = layer.project(x)
    o = nv.gdn_prefill(*parts, state, cu, state_index=index)
    ys = [layer.out(o)]
    torch.cuda.synchronize()
    _check(parts, ends, None, start, o, state, [2, 0])
    assert torch.equal(state[1], start[1])
    for t in range(steps):
        before = state.clone()
        parts = layer.project(xs[t])
        o = nv.gdn_step(*parts, state, state_index=index)
        ys.append(layer.out(o))
        torch.cuda.synchronize()
        _check(parts, np.arange(3), np.ones(2), before, o, state, [2, 0])
        assert torch.equal(state[1], start[1])
    assert all(torch.isfinite(y).all() and y.abs().max() > 0 for y in ys)

    # one captured step, replayed: the same six tokens from the same states, eager work between
    again, one = start.clone(), xs[0].clone()
    nv.gdn_prefill(*layer.project(x), again, cu, state_index=index)
    torch.cuda.synchronize()
    kept = again.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.out(nv.gdn_step(*layer.project(one), again, state_index=index))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.out(nv.gdn_step(*layer.project(one), again, state_index=index))
    again.copy_(kept)
    for t in range(steps):
        one.copy_(xs[t])
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        (torch.ones(8, device=DEV) * 2).sum().item()
        torch.cuda.synchronize()
        assert torch.equal(y, ys[1 + t]), f"replay {t}"
    assert torch.equal(again, state)


def test_calls_by_name_equal_calls_by_place():
    g = torch.Generator(DEV).manual_seed(3)
    rows = lambda n, h: torch.randn(n, h, D, device=DEV, generator=g).bfloat16()  # noqa: E731
    slots = torch.arange(40, device=DEV)
    q, k, v = rows(40, 8), rows(40, 2), rows(40, 2)
    caches = [nv.PagedKVCache.empty(4, 16, 2, D, DEV) for _ in range(2)]
    for c in caches:
        c.k.zero_(), c.v.zero_()
    a = nv.kv_append(k, v, caches[0], slots, q)
    b = nv.kv_append(k=k, v=v, cache=caches[1], slots=slots, q=q)
    assert torch.equal(a, b) and torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    table, lens = torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), torch.tensor([40], dtype=torch.int32, device=DEV)
    x = nv.attn_decode(q[:1], caches[0], table, lens)
    y = nv.attn_decode(q=q[:1], cache=caches[0], block_table=table, seq_lens=lens, stream=torch.cuda.current_stream())
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    layer = Recurrent(4)
    parts = layer.project(torch.randn(40, WIDTH, device=DEV, generator=g).bfloat16())
    named = dict(zip("qkvg", parts), beta=parts[4])
    cu = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    s, t = (torch.zeros(40, HV, D, D, device=DEV) for _ in range(2))
    assert torch.equal(nv.gdn_prefill(*parts, s, cu), nv.gdn_prefill(**named, state=t, cu_seqlens=cu)) and torch.equal(s, t)
    assert torch.equal(nv.gdn_step(*parts, s), nv.gdn_step(**named, state=t)) and torch.equal(s, t)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_past_two_to_the_31st_element(fp8):
    """Pages of a pool of more than 2^31 elements, short and split sequences: the same as from a
    small pool that holds the same rows."""
    pages, page, kv = 16500, 128, 8                       # 2.16e9 elements
    say(f"[layers] attention in a pool of {pages * page * kv * D} elements fp8={fp8}")
    g = torch.Generator(DEV).manual_seed(6)
    amax = [torch.tensor([4.0], device=DEV) for _ in range(2)] if fp8 else [None, None]
    big, small = nv.PagedKVCache.empty(pages, page, kv, D, DEV, *amax), nv.PagedKVCache.empty(40, page, kv, D, DEV, *amax)
    far = pages - 1 - 2 * torch.randperm(40, device=DEV, generator=g)
    for a, b in ((big.k, small.k), (big.v, small.v)):
        if fp8:
            b.random_(0, 0x70, generator=g)
        else:
            b.normal_(generator=g)
        a[far] = b
    table = torch.arange(40, device=DEV).view(2, 20)
    lens = torch.tensor([20 * page - 3, 300], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 16, D, device=DEV, generator=g).bfloat16()
    for bound in (20 * page, 512):
        n = lens.clamp_max(bound)
        x = nv.attn_decode(q, big, far[table].int(), n, max_len=bound)
        y = nv.attn_decode(q, small, table.int(), n, max_len=bound)
        torch.cuda.synchronize()
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]) and torch.isfinite(x[1]).all()
