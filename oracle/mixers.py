"""The token mixers in plain form (CPU oracle): rotation and paged append bit for bit,
decode attention and the gated delta rule in binary64.

TEST INFRASTRUCTURE ONLY -- see the package docstring for who may use it.

  * append: fl(fl(x1 c) - fl(x2 s)), fl(fl(x2 c) + fl(x1 s)) in binary32, bf16 RNE, then
    the cache codec of oracle/kvfp8.py for an E4M3 cache;
  * attention: softmax(scale q K^T) V over the last `window` of the first `len` cached
    tokens, the tokens of pages outside the pool left out; zeros and -inf for no token;
  * gated delta rule: S <- e^g S, u = beta (v - S^T k), S <- S + k u^T, o = scale S^T q,
    without beta u = v.
"""
import numpy as np

from . import kvfp8


def bf16_bits(v):
    return kvfp8.bf16_bits_of_f32(v)


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def rotate(x, cos, sin, interleaved):
    """float32 [..., dim]; cos, sin float32 [..., rot / 2]: the first rot elements in pairs."""
    half = cos.shape[-1]
    y = np.array(x, np.float32)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., first].copy(), y[..., second].copy()
    with np.errstate(all="ignore"):
        y[..., first] = a * cos - b * sin
        y[..., second] = b * cos + a * sin
    return y


def append(q, k, v, rope, rot, interleaved, positions, slots, k_pool, v_pool, q_out, k_amax=None, v_amax=None):
    """Updates k_pool, v_pool (uint8 codes or uint16 bf16 bits, [pages, page, heads, dim]) and
    q_out (uint16 bits) in place, token by token.  q, k, v: float32 [T, heads, dim]."""
    pages, page = k_pool.shape[:2]
    for t, slot in enumerate(slots):
        if slot < 0 or slot >= pages * page:
            continue
        kt, qt = k[t], None if q is None else q[t]
        if rot:
            if positions[t] < 0 or positions[t] >= rope.shape[0]:
                continue
            cos, sin = rope[positions[t], : rot // 2], rope[positions[t], rot // 2:]
            kt = rotate(kt, cos, sin, interleaved)
            qt = None if q is None else rotate(qt, cos, sin, interleaved)
        if q is not None:
            q_out[t] = bf16_bits(qt)
        for pool, x, amax in ((k_pool, kt, k_amax), (v_pool, v[t], v_amax)):
            bits = bf16_bits(x)
            pool[slot // page, slot % page] = bits if amax is None else kvfp8.encode(bf16_value(bits), np.float32(amax))


def attend(q, k_pool, v_pool, table, lens, max_len, scale, window, kv_heads):
    """float64 out [B, H, D], lse [B, H], and sum p |v| (the scale of out's errors) and the largest
    score bound scale * sum |q||k| for the tests' tolerances.  q: [B, H, D]; pools: float64
    [pages, page, kv_heads, D]."""
    B, H, D = q.shape
    pages, page = k_pool.shape[:2]
    out, lse, mag, top = np.zeros((B, H, D)), np.full((B, H), -np.inf), np.zeros((B, H, D)), np.zeros((B, H))
    for b in range(B):
        n = min(max(int(lens[b]), 0), max_len)
        at = np.arange(max(0, n - window) if window else 0, n)
        p = table[b][at // page] if len(at) else at
        at, p = at[(p >= 0) & (p < pages)], p[(p >= 0) & (p < pages)]
        if len(at) == 0:
            continue
        for h in range(H):
            kk, vv = (x[p, at % page, h // (H // kv_heads)] for x in (k_pool, v_pool))
            s = scale * (kk @ q[b, h])
            m = s.max()
            e = np.exp(s - m)
            out[b, h], mag[b, h] = (e @ vv) / e.sum(), (e @ np.abs(vv)) / e.sum()
            lse[b, h], top[b, h] = m + np.log(e.sum()), (abs(scale) * (np.abs(kk) @ np.abs(q[b, h]))).max()
    return out, lse, mag, top


def recur(q, k, v, g, beta, S, scale):
    """One sequence, one head: q, k [T, Dk], v [T, Dv], g, beta [T], S [Dk, Dv] (float64) ->
    out [T, Dv], the last state, and the largest norm of any state on the way."""
    S = np.array(S, np.float64)
    out, largest = np.zeros(v.shape), np.linalg.norm(S)
    for t in range(q.shape[0]):
        S *= np.exp(g[t])
        u = v[t] if beta is None else beta[t] * (v[t] - k[t] @ S)
        S += np.outer(k[t], u)
        out[t] = scale * (q[t] @ S)
        largest = max(largest, np.linalg.norm(S))
    return out, S, largest


def gdn(q, k, v, g, beta, state, index, ends, has, scale):
    """The layer: q, k [T, Hk, Dk], v [T, Hv, Dv], g, beta [T, Hv], state [N, Hv, Dk, Dv] float64;
    ends: B + 1 row bounds.  Returns out (NaN where nothing is written), states, and norms [N, Hv]."""
    state = np.array(state, np.float64)
    out, norms = np.full(v.shape, np.nan), np.zeros(state.shape[:2])
    many = v.shape[1] // q.shape[1]
    for b in range(len(ends) - 1):
        slot = b if index is None else int(index[b])
        if slot < 0 or slot >= len(state):
            continue
        r = slice(ends[b], ends[b + 1])
        for h in range(v.shape[1]):
            first = state[slot, h] if has is not None and has[b] else np.zeros_like(state[slot, h])
            out[r, h], state[slot, h], norms[slot, h] = recur(
                q[r, h // many], k[r, h // many], v[r, h], g[r, h], None if beta is None else beta[r, h], first, scale)
    return out, state, norms
