"""Drafted tokens in plain form (CPU oracle), in binary64: the norm of a head, attention of a
tree of drafted tokens, the verification of drafts, and cache rows and pages that move.

TEST INFRASTRUCTURE ONLY -- see the package docstring for who may use it.
"""
import numpy as np


def norm(x, w, eps):
    """float64 [..., dim]: x / sqrt(mean(x^2) + eps) * w; zeros for a head of zeros where eps is 0."""
    with np.errstate(all="ignore"):
        return np.nan_to_num(x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)) * w


def way(parents, i):
    """The nodes from the context down to node i (ascending, i last); [] for a padded node.  None: a chain."""
    if parents is None:
        return list(range(i + 1))
    nodes = [i]
    while True:
        up = int(parents[nodes[-1]])
        if up == -1:
            return nodes[::-1]
        if not 0 <= up < nodes[-1]:
            return []
        nodes.append(up)


def seen(parents, i, ctx, window):
    """Rows of the sequence that node i attends to, in order."""
    nodes = way(parents, i)
    if not nodes:
        return np.zeros(0, np.int64)
    rows = np.concatenate([np.arange(ctx), ctx + np.array(nodes)]).astype(np.int64)
    return rows[-window:] if window else rows


def attend(q, k_pool, v_pool, table, ctx_lens, parents, max_len, scale, window, kv_heads):
    """q: [B, W, H, D]; pools: float64 [pages, page, kv_heads, D].  Returns out, lse, and for the tests'
    tolerances sum p |v| and the largest scale * sum |q||k| (see oracle/mixers.py)."""
    B, W, H, D = q.shape
    pages, page = k_pool.shape[:2]
    out, lse, mag, top = np.zeros((B, W, H, D)), np.full((B, W, H), -np.inf), np.zeros((B, W, H, D)), np.zeros((B, W, H))
    for b in range(B):
        ctx = min(max(int(ctx_lens[b]), 0), max_len)
        for i in range(W):
            at = seen(None if parents is None else parents[b], i, ctx, window)
            p = table[b][at // page]
            at, p = at[(p >= 0) & (p < pages)], p[(p >= 0) & (p < pages)]
            if len(at) == 0:
                continue
            for g in range(kv_heads):
                kk, vv = (x[p, at % page, g] for x in (k_pool, v_pool))
                hs = slice(g * (H // kv_heads), (g + 1) * (H // kv_heads))
                s = scale * (q[b, i, hs] @ kk.T)
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                n = e.sum(-1, keepdims=True)
                out[b, i, hs], mag[b, i, hs] = (e @ vv) / n, (e @ np.abs(vv)) / n
                lse[b, i, hs] = (m + np.log(n))[:, 0]
                top[b, i, hs] = (abs(scale) * (np.abs(q[b, i, hs]) @ np.abs(kk).T)).max(-1)
    return out, lse, mag, top


def softmax(x, t):
    with np.errstate(all="ignore"):
        e = np.exp((x.astype(np.float64) - x.max()) / t)
        return e / e.sum()


def verify(logits, drafts, parents, temperature, uniforms, draft_logits=None):
    """One sequence: logits float32 [W, V], drafts [W], parents [W] or None, temperature (0: greedy), uniforms
    [W + 1] -> (tokens, path, margin): margin is how far the closest decision is from its border, in probability."""
    W, V = logits.shape
    up = list(range(-1, W - 1)) if parents is None else [int(p) for p in parents]
    if up[0] != -1:
        return [], [], 1.0
    node, tokens, path, margin = 0, [], [0], 1.0
    while True:
        row = logits[node]
        kids = [c for c in range(node + 1, W) if up[c] == node and 0 <= drafts[c] < V]
        taken, largest = None, int(np.argmax(row)) if row.max() > -np.inf else -1
        if not temperature > 0:
            taken = next((c for c in kids if drafts[c] == largest), None)
        elif row.max() > -np.inf:
            weights = softmax(row, temperature)
            u = float(uniforms[node])
            if draft_logits is not None:
                if kids:
                    x = int(drafts[kids[0]])
                    q = softmax(draft_logits[node], temperature)
                    margin = min(margin, abs(u * q[x] - weights[x]))
                    if u * q[x] < weights[x]:
                        taken = kids[0]
                    else:
                        weights = np.maximum(weights - q, 0)
            else:
                total, tried = 0.0, []
                for c in kids:
                    if drafts[c] in tried:
                        continue
                    tried.append(int(drafts[c]))
                    total += weights[drafts[c]]
                    margin = min(margin, abs(u - total))
                    if u < total:
                        taken = c
                        break
                else:
                    weights = weights.copy()
                    weights[tried] = 0
        else:
            weights = np.zeros(V)
        if taken is None:
            break
        node = taken
        path.append(node)
        tokens.append(int(drafts[node]))
    last = largest
    if temperature > 0 and weights.sum() > 0:
        run = np.cumsum(weights)
        target = float(uniforms[W]) * run[-1]
        last = int(np.searchsorted(run, target, side="right"))
        margin = min(margin, np.abs(run - target).min() if target > 0 else 1.0)
    return tokens + [last], path, margin


def compact(pools, table, ctx_lens, path, counts):
    """Moves rows of pools [pages, page, ...] in place: row ctx + path[i] to ctx + i for i < counts."""
    pages, page = pools[0].shape[:2]
    W = path.shape[1]
    for b in range(len(ctx_lens)):
        moves = []
        for i in range(min(max(int(counts[b]), 0), W)):
            j, ctx = int(path[b, i]), int(ctx_lens[b])
            if j == i or not 0 <= j < W or ctx < 0 or ctx + max(i, j) >= table.shape[1] * page:
                continue
            src, dst = ((int(table[b, r // page]), r % page) for r in (ctx + j, ctx + i))
            if 0 <= src[0] < pages and 0 <= dst[0] < pages:
                moves.append((src, dst))
        for p in pools:
            rows = [p[s].copy() for s, _ in moves]
            for (_, d), r in zip(moves, rows):
                p[d] = r


def copy_pages(pools, src, dst):
    """Copies pages of pools [pages, ...] in place."""
    for p in pools:
        for s, d in zip(src, dst):
            if 0 <= s < len(p) and 0 <= d < len(p):
                p[d] = p[s]
