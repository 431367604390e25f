"""GPU parity of the paged cache append, bit for bit against oracle/mixers.py: both source and
cache types, both pair layouts, partial and no rotation, cache layouts, padded rows, slots and
positions out of range, strided inputs, one token and many."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
import workloads as W
from gpu_util import DEV, say
from oracle import mixers as M

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _pools(pages, page, kv, dim, fp8, layout, seed):
    rng = np.random.default_rng(seed)
    raw = [rng.integers(0, 0x78, (pages, page, kv, dim)).astype(np.uint8 if fp8 else np.uint16) for _ in range(2)]
    dt = torch.uint8 if fp8 else torch.bfloat16
    dev = [torch.from_numpy(r if fp8 else r.view(np.int16)).to(DEV).view(dt) for r in raw]
    if layout == "side by side":            # [pages, 2, page, kv, dim]
        both = torch.stack(dev, 1)
        dev = [both[:, 0], both[:, 1]]
    elif layout == "heads first":           # [pages, kv, page, dim]
        dev = [d.transpose(1, 2).contiguous().transpose(1, 2) for d in dev]
    return raw, dev


def _values(t, fp8):
    return t.cpu().numpy() if fp8 else _bits(t).reshape(t.shape)


def check(T, heads, kv, dim, rot, inter, page, src, fp8, layout="plain", pad=0, strided=False, with_q=True, seed=0):
    say(f"[append] T={T} heads={heads}/{kv}x{dim} rot={rot} inter={inter} page={page} {src} fp8={fp8} {layout} pad={pad}")
    rng = np.random.default_rng(seed + T)
    width = (heads + 2 * kv) * dim
    x = (rng.standard_normal((T, width)) * rng.choice([1.0, 30.0], width, p=[0.97, 0.03])).astype(np.float32)
    dt = torch.float32 if src == "f32" else torch.bfloat16
    fused = torch.from_numpy(x).to(dt).to(DEV)
    x = fused.float().cpu().numpy()
    if not strided:
        parts = [p.contiguous() for p in fused.split([heads * dim, kv * dim, kv * dim], 1)]
    else:
        parts = fused.split([heads * dim, kv * dim, kv * dim], 1)
    q, k, v = (p.view(T, p.shape[1] // dim, dim) for p in parts)
    xs = [a.reshape(T, a.shape[1] // dim, dim) for a in np.split(x, [heads * dim, (heads + kv) * dim], 1)]
    far = 4096
    ang = np.arange(far)[:, None] / 1e4 ** (np.arange(0, rot, 2) / max(rot, 1)) if rot else np.zeros((far, 0))
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    pos = rng.integers(0, far, T).astype(np.int64)
    if pad:
        slots[-pad:] = -1
        if T > 3 * pad:
            slots[0], slots[1] = pages * page, -(1 << 40)
            pos[2], pos[3] = far, -1
    raw, dev = _pools(pages, page, kv, dim, fp8, layout, seed)
    amax = [np.float32(5.3), np.float32(0.0 if seed == 9 else 7.1)] if fp8 else [None, None]
    q_ref = np.full((T, heads, dim), 0x1234, np.uint16)
    q_out = torch.from_numpy(q_ref.view(np.int16).copy()).to(DEV).view(torch.bfloat16)
    M.append(xs[0] if with_q else None, xs[1], xs[2], rope, rot, inter, pos, slots, raw[0], raw[1], q_ref, *amax)
    cache = nv.PagedKVCache(dev[0], dev[1], *[None if a is None else torch.tensor([a], device=DEV) for a in amax])
    to = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    got = nv.kv_append(k, v, cache, to(slots), q=q if with_q else None, positions=to(pos) if rot else None,
                       rope=to(rope) if rot else None, interleaved=inter, q_out=q_out if with_q else None)
    torch.cuda.synchronize()
    assert (got is None) == (not with_q)
    assert np.array_equal(_values(dev[0], fp8), raw[0]), "keys differ"
    assert np.array_equal(_values(dev[1], fp8), raw[1]), "values differ"
    assert np.array_equal(_bits(q_out).reshape(q_ref.shape), q_ref), "queries differ"


@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,heads,kv,dim,rot,inter,page", [
    (1, 40, 8, 128, 128, False, 64), (133, 24, 4, 256, 64, True, 16), (37, 16, 16, 64, 32, False, 48),
    (70, 5, 1, 128, 16, True, 16), (19, 3, 3, 64, 0, False, 32)])
def test_append(T, heads, kv, dim, rot, inter, page, src, fp8):
    check(T, heads, kv, dim, rot, inter, page, src, fp8, strided=T % 2 == 1, pad=0 if T == 1 else 4)


@pytest.mark.parametrize("layout", ["side by side", "heads first"])
@pytest.mark.parametrize("fp8", [False, True])
def test_cache_layouts(layout, fp8):
    check(50, 8, 2, 128, 128, False, 16, "f32", fp8, layout=layout, pad=3, strided=True)


def test_without_queries_and_zero_amax():
    check(21, 8, 2, 64, 64, False, 16, "bf16", True, with_q=False, seed=9)


def test_only_padding_and_no_tokens():
    check(5, 8, 2, 64, 64, False, 16, "f32", True, pad=5)
    check(0, 8, 2, 64, 64, False, 16, "f32", False)


def test_agrees_with_the_codec():
    """Values go through nvfp4_kv_fp8_encode's steps: the same codes as the codec's own call."""
    T, kv, dim = 64, 8, 128
    v = W.bf16_bits(np.random.default_rng(5).standard_normal((T, kv * dim)).astype(np.float32))
    v = torch.from_numpy(v.view(np.int16)).to(DEV).view(torch.bfloat16)
    amax = torch.tensor([3.0], device=DEV)
    cache = nv.PagedKVCache.empty(1, 64, kv, dim, DEV, amax, amax)
    x = v.view(T, kv, dim)
    nv.kv_append(x, x, cache, torch.arange(T, device=DEV))
    assert torch.equal(cache.k.view(T, -1), nv.kv_fp8_encode(v, amax)) and torch.equal(cache.k, cache.v)


def test_rows_past_two_to_the_31st_element():
    """A pool of more than 2^31 elements: the last page's rows land where they belong."""
    pages, page, kv, dim = 16500, 128, 8, 128          # 2.16e9 elements of one byte
    amax = torch.tensor([4.0], device=DEV)
    cache = nv.PagedKVCache.empty(pages, page, kv, dim, DEV, amax, amax)
    cache.k[-1].zero_(), cache.v[-1].zero_()
    x = torch.randn(3, kv, dim, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16()
    slots = torch.tensor([pages * page - 1, pages * page - 128, pages * page - 60], device=DEV)
    nv.kv_append(x, -x, cache, slots)
    ref = nv.kv_fp8_encode(x, amax)
    rows = slots - (pages - 1) * page
    assert torch.equal(cache.k[-1][rows], ref) and torch.equal(cache.v[-1][rows], ref ^ 0x80)
