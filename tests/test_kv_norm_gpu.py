"""The append with a norm of each head against oracle/drafts.py in 64 bits.

Tolerance.  The squares' sum of D elements is taken by additions of at most 16 + 4 terms one after
the other, each rounding by 2^-24; the square root halves that; with the mean, eps, the root, the
quotient and two products the normed value y is off by at most 16 * 2^-24 |y|.  A rotated element is
a sum of two products, 2 * 2^-24 of each more.  Then one rounding to bf16 (2^-8 of the value).  A code of
the E4M3 cache stands for E4M3(bf16 * gain): its own rounding is 2^-4 of the value, or half of the
smallest step, 2^-10."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import drafts as O
from oracle import kvfp8 as F
from oracle import mixers as M

pytestmark = pytest.mark.gpu


def _rotate(y, cos, sin, inter):
    """Rotated values and the sum of the two products' magnitudes, float64 [T, H, D]."""
    z, mag = y.copy(), np.abs(y)
    half = cos.shape[1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    c, s = cos[:, None].astype(np.float64), sin[:, None].astype(np.float64)
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    mag[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
    mag[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return z, mag


def check(T, heads, kv, dim, rot, inter, src, fp8, norms="qk", eps=1e-6, strided=False, with_q=True, seed=0, zero=False):
    say(f"[norm] T={T} heads={heads}/{kv}x{dim} rot={rot} inter={inter} {src} fp8={fp8} norms={norms} eps={eps}")
    rng = np.random.default_rng(seed + T + dim)
    width, page, far = (heads + 2 * kv) * dim, 16, 300
    x = rng.standard_normal((T, width)) * rng.choice([1.0, 30.0, 1e-4], width, p=[0.9, 0.05, 0.05])
    x *= rng.choice([1.0, 1e-6, 1e8], (T, 1))
    if zero:
        x[0] = 0
    fused = torch.from_numpy(x.astype(np.float32)).to(torch.float32 if src == "f32" else torch.bfloat16).to(DEV)
    x = fused.double().cpu().numpy()
    parts = fused.split([heads * dim, kv * dim, kv * dim], 1)
    q, k, v = ((p if strided else p.contiguous()).view(T, -1, dim) for p in parts)
    xq, xk, xv = (a.reshape(T, -1, dim) for a in np.split(x, [heads * dim, (heads + kv) * dim], 1))
    wq, wk = ((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2))
    ang = np.arange(far)[:, None] / 1e4 ** (np.arange(0, rot, 2) / max(rot, 1))
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pages = -(-T // page) + 1
    slots, pos = rng.permutation(pages * page)[:T], rng.integers(0, far, T)
    if T > 2:
        slots[1] = -1
    amax = [torch.tensor([a], device=DEV) for a in (9.0, 7.0)] if fp8 else [None, None]
    cache = nv.PagedKVCache.empty(pages, page, kv, dim, DEV, *amax)
    cache.k.view(torch.uint8).fill_(0x11), cache.v.view(torch.uint8).fill_(0x11)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    q_out = torch.full((T, heads, dim), 5.0, device=DEV).bfloat16()
    got = nv.kv_append(k, v, cache, to(slots), q=q if with_q else None, positions=to(pos) if rot else None,
                       rope=to(rope) if rot else None, interleaved=inter, q_out=q_out if with_q else None,
                       q_norm=to(wq) if "q" in norms and with_q else None, k_norm=to(wk) if "k" in norms else None, eps=eps)
    torch.cuda.synchronize()
    assert (got is None) == (not with_q)
    ok = slots >= 0
    cos, sin = rope[pos][:, : rot // 2], rope[pos][:, rot // 2:]
    yq, mq = _rotate(O.norm(xq, wq, eps) if "q" in norms else xq, cos, sin, inter)
    yk, mk = _rotate(O.norm(xk, wk, eps) if "k" in norms else xk, cos, sin, inter)
    if with_q:
        out = got.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(yq) + 20 * 2.0 ** -24 * mq + 1e-38
        assert (np.abs(out - yq) <= tol)[ok].all(), f"queries: {(np.abs(out - yq) / tol)[ok].max():.3f} of the tolerance"
        assert (out[~ok] == 5.0).all()
    # values are not normed: bit for bit
    rows = cache.v.view(-1, kv, dim)[to(slots[ok])].cpu()
    bits = M.bf16_bits(xv[ok].astype(np.float32))
    if fp8:
        assert np.array_equal(rows.numpy(), F.encode(M.bf16_value(bits), np.float32(7.0)))
    else:
        assert np.array_equal(rows.contiguous().view(torch.int16).numpy().view(np.uint16), bits)
    rows = cache.k.view(-1, kv, dim)[to(slots[ok])].cpu()
    tol = (2.0 ** -8 * np.abs(yk) + 20 * 2.0 ** -24 * mk + 1e-38)[ok]
    if fp8:
        gain = float(np.float32(448.0) / np.float32(9.0))
        ref = np.clip(yk[ok] * gain, -448, 448)
        val = F.decode_f32(rows.numpy(), 448.0).astype(np.float64)
        tol = tol * gain * (1 + 2.0 ** -4) + 2.0 ** -4 * np.abs(ref) + 2.0 ** -10
    else:
        ref, val = yk[ok], rows.double().numpy()
    assert (np.abs(val - ref) <= tol).all(), f"keys: {(np.abs(val - ref) / tol).max():.3f} of the tolerance"
    untouched = np.ones(pages * page, bool)
    untouched[slots[ok]] = False
    for t in (cache.k, cache.v):
        assert (t.view(torch.uint8).view(pages * page, -1)[to(untouched)] == 0x11).all()


@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,heads,kv,dim,rot,inter", [
    (1, 40, 8, 128, 128, False), (133, 24, 4, 256, 64, True), (37, 16, 16, 64, 32, False), (70, 5, 1, 128, 16, True),
    (19, 3, 3, 64, 0, False), (9, 33, 11, 256, 256, False)])
def test_norms(T, heads, kv, dim, rot, inter, src, fp8):
    check(T, heads, kv, dim, rot, inter, src, fp8, strided=T % 2 == 1)


@pytest.mark.parametrize("norms", ["q", "k"])
def test_one_norm_only(norms):
    check(20, 8, 2, 128, 64, False, "f32", False, norms=norms)


def test_without_queries_and_with_zeros():
    check(21, 8, 2, 64, 64, False, "bf16", True, with_q=False)
    check(5, 8, 2, 64, 64, False, "f32", False, eps=0.0, zero=True)
    check(5, 8, 2, 128, 64, True, "f32", False, eps=1e-3, zero=True)


def test_no_tokens():
    cache = nv.PagedKVCache.empty(1, 16, 2, 64, DEV)
    x, w = torch.empty(0, 2, 64, device=DEV), torch.ones(64, device=DEV)
    q = nv.kv_append(x, x, cache, torch.empty(0, dtype=torch.int64, device=DEV), q=torch.empty(0, 4, 64, device=DEV), q_norm=w, k_norm=w)
    assert q.shape == (0, 4, 64)


def test_without_weights_it_is_the_plain_append():
    """nvfp4_kv_append_norm without weights: nvfp4_kv_append, bit for bit."""
    g = torch.Generator(DEV).manual_seed(3)
    k, q = torch.randn(9, 2, 64, device=DEV, generator=g), torch.randn(9, 4, 64, device=DEV, generator=g)
    slots = torch.arange(9, device=DEV)
    a, b = (nv.PagedKVCache.empty(1, 16, 2, 64, DEV) for _ in range(2))
    x = nv.kv_append(k, k, a, slots, q=q)
    y = torch.empty_like(x)
    nv.nvfp4_kv_append_norm(q, k, k, 0, 9, 4, 256, 128, 128, None, None, 1e-6, None, 0, 0, False, None, slots, b.desc, y, 256)
    torch.cuda.synchronize()
    assert torch.equal(x, y) and torch.equal(a.k[0, :9], b.k[0, :9]) and torch.equal(a.v[0, :9], b.v[0, :9])
