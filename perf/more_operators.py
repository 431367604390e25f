"""Speculative decoding over the paged key-value cache, as workloads: the append with a norm for each
head, attention for a tree of drafted tokens, the verification of the drafts, and the cache rows and
pages that move afterwards.

Each workload has a plain form in elementary torch operations and the call of the library that does
the same work; `own` says which of the two `run` takes.  Head counts and cache sizes are those of this
repository's workloads (8 key-value heads of 128 beside 5120 channels, a 32768-token cache of 1024
channels, 16 attention layers); vocabularies and trees are generic.

Definitions (the plain forms below are their direct transcription):

  append   Each head of q and k: y = x * w / sqrt(mean(x^2) + eps); its first `rot` elements are then
           rotated by the angle of the token's position (fp32 tables of cos and sin; pairs (i, i + rot/2),
           or (2i, 2i + 1) interleaved), rounded to bf16, and k and v go to the cache row `slot`: as bf16,
           or as E4M3 codes of x * fl(448 / amax).  A negative slot marks a padded row: nothing is written.
  attend   Sequence b has ctx[b] cached tokens, and behind them `nodes` drafted ones whose keys and values
           are in the cache too.  Node i has the parent parents[b][i] (-1: the context itself; anything but
           -1 .. i - 1, also anywhere on the way up: a padded node).  It sees the context, its ancestors
           and itself, of all these in order the last `window` (all if 0):
           out = sum_j softmax_j(scale * q . K_j) V_j, lse the softmax's log sum; zeros and -inf for a padded node.
  verify   Node 0 is the last token known, node i > 0 the drafted token drafts[b][i]; logits[b][i] are the
           target model's after node i, p_i = softmax(logits[b][i] / temperature[b]).  From node 0 on:
           without draft logits, the children c of the node i that is reached, in order, each token once:
           the first with uniforms[b][i] < sum of p_i over the children up to it is accepted; with draft
           logits (q_i = softmax(draft_logits[b][i] / temperature[b])) the first child alone, if
           uniforms[b][i] q_i(x) < p_i(x); at temperature 0 the first child that is p_i's largest.
           Where no child is accepted a last token is drawn with uniforms[b][nodes], the first whose running
           sum of weights is above uniforms[b][nodes] times their sum: the weights are p_i without the children's
           tokens, with draft logits max(p_i - q_i, 0), at a node without children p_i; the largest at temperature 0.
           tokens: the accepted ones and the last; path: the accepted nodes, node 0 first; counts: their number.
  compact  Cache row ctx[b] + path[b][i] moves to row ctx[b] + i, for i < counts[b], in every layer.
  copy     Page src[i] is copied to page dst[i], in every layer.
"""
import math
import random

import torch

own = False
DEV = "cuda:0"
MAX_NODES = 64


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    """Smallest, ordinary and largest call of each operator."""
    append = dict(op="append", heads=40, kv=8, dim=128, rot=128, inter=False, page=64, pad=0)
    attend = dict(op="attend", heads=40, kv=8, dim=128, page=64, window=0, pad=0, chain=False)
    verify = dict(op="verify", sampled=False, greedy=0)
    move = dict(kv=8, dim=128, page=64, cache="fp8", layers=16)
    return [
        # one request's tree of eight drafted tokens: the rows of the fused fp32 projection go to an FP8 cache
        dict(append, name="append_8_f32_fp8", tokens=8, src="f32", cache="fp8"),
        # a whole 32768-token prompt of the 8 x 128 cache
        dict(append, name="append_32768_f32_fp8", tokens=32768, src="f32", cache="fp8"),
        # one chat turn of one request with a chain of five tokens: latency
        dict(attend, name="attend_1x5_1021_fp8", batch=1, nodes=5, longest=1021, cache="fp8", chain=True),
        # an ordinary serving batch of uneven lengths, trees of 16, two padded sequences
        dict(attend, name="attend_48x16_4099_fp8", batch=48, nodes=16, longest=4099, cache="fp8", pad=2),
        # few long documents, the widest trees, wide heads, bf16 cache: as much matrix work as a prompt's
        dict(attend, name="attend_6x64_32768_bf16", batch=6, nodes=64, longest=32768, cache="bf16", heads=24, kv=4, dim=256, page=128),
        # one request, eight nodes, a small vocabulary: latency
        dict(verify, name="verify_1x8_32000", batch=1, nodes=8, vocab=32000),
        # a batch of chains drawn from a draft model's own distribution, a vocabulary that divides by nothing
        dict(verify, name="verify_29x6_100003_sampled", batch=29, nodes=6, vocab=100003, sampled=True),
        # a full batch of trees, some sequences greedy
        dict(verify, name="verify_64x24_131072", batch=64, nodes=24, vocab=131072, greedy=5),
        # the accepted rows of one request, and of a batch, in all attention layers
        dict(move, name="compact_1x8", op="compact", batch=1, nodes=8, longest=1021),
        dict(move, name="compact_64x24", op="compact", batch=64, nodes=24, longest=200),
        # the last page of a prompt that three answers go on from
        dict(move, name="copy_3", op="copy", pages=3, pool=12),
        # a batch of prompts forked as a whole
        dict(move, name="copy_96", op="copy", pages=96, pool=200),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case: sizes spread over their logarithm, the operators in turn by chance."""
    op = rng.choice(["append", "attend", "attend", "verify", "verify", "compact", "copy"])
    shapes = [(40, 8, 128), (32, 8, 128), (24, 4, 256), (16, 16, 64), (48, 2, 128)]
    if op == "append":
        heads, kv, dim = rng.choice(shapes)
        tokens = _log(rng, 1, 24000)
        return dict(op=op, heads=heads, kv=kv, dim=dim, rot=rng.choice([dim, dim // 2, 32]), inter=rng.random() < 0.3,
                    page=rng.choice([16, 48, 64, 128]), pad=rng.choice([0, 0, min(tokens - 1, 7)]), tokens=tokens,
                    src=rng.choice(["f32", "bf16"]), cache=rng.choice(["fp8", "bf16"]))
    if op == "attend":
        heads, kv, dim = rng.choice(shapes)
        batch, nodes = _log(rng, 1, 96), _log(rng, 1, MAX_NODES)
        most = min(32768, 131072 * 1024 // (batch * kv * dim), 4 * 64 * 24 * 32768 * 256 // (batch * nodes * heads * dim))
        longest = _log(rng, 16, max(17, most))
        return dict(op=op, heads=heads, kv=kv, dim=dim, page=rng.choice([16, 48, 64, 128]),
                    window=rng.choice([0, 0, max(1, longest // 3)]), batch=batch, nodes=nodes, longest=longest,
                    cache=rng.choice(["fp8", "bf16"]), pad=rng.choice([0, min(batch - 1, 3)]), chain=rng.random() < 0.3)
    if op == "verify":
        vocab = rng.choice([32000, 50257, 65536, 100003, 131072])
        batch, sampled = _log(rng, 1, 96), rng.random() < 0.4
        nodes = _log(rng, 1, min(MAX_NODES, max(2, (96 << 20) // (batch * vocab))))
        return dict(op=op, batch=batch, nodes=nodes, vocab=vocab, sampled=sampled, greedy=rng.choice([0, 0, batch // 3]))
    kv, dim = rng.choice([(8, 128), (4, 256), (16, 64), (2, 128)])
    c = dict(op=op, kv=kv, dim=dim, page=rng.choice([16, 48, 64, 128]), cache=rng.choice(["fp8", "bf16"]), layers=rng.randint(1, 16))
    if op == "compact":
        return dict(c, batch=_log(rng, 1, 48), nodes=_log(rng, 2, 24), longest=_log(rng, 16, 400))
    pages = _log(rng, 1, 64)
    return dict(c, page=rng.choice([16, 48, 64]), pages=pages, pool=2 * pages + rng.randint(1, 9))


def _lengths(batch, longest, pad=0):
    """Uneven lengths of a batch, one of them the longest; `pad` empty ones at its end."""
    r = random.Random(batch * 1000003 + longest)
    n = [r.randint(max(1, longest // 4), longest) for _ in range(batch)]
    n[r.randrange(batch - pad)] = longest
    return n[: batch - pad] + [0] * pad if pad else n


def _parents(r, nodes, chain):
    """A tree as drafters grow it: mostly on from the newest nodes; the last few nodes of some are padding."""
    if chain:
        return list(range(-1, nodes - 1))
    tree = [-1] + [i - 1 - int(r.random() ** 2 * min(i, 6)) for i in range(1, nodes)]
    for i in range(nodes - r.choice([0, 0, nodes // 4]), nodes):
        tree[i] = -2
    return tree


def work(case):
    c = case
    size = 1 if c.get("cache") == "fp8" else 2
    if c["op"] == "append":
        t, src = c["tokens"] - c["pad"], 4 if c["src"] == "f32" else 2
        q, kv = c["heads"] * c["dim"], 2 * c["kv"] * c["dim"]
        table = 4 * c["rot"] + 16
        return {"bytes": t * ((q + kv) * src + 2 * q + kv * size + table),
                "flops": t * (c["heads"] + c["kv"]) * (3 * c["rot"] + 4 * c["dim"])}
    if c["op"] == "attend":
        n = [min(x, c["window"]) if c["window"] else x for x in _lengths(c["batch"], c["longest"], c["pad"])]
        cached, rows = sum(n) + (c["batch"] - c["pad"]) * c["nodes"], c["batch"] * c["nodes"] * c["heads"]
        return {"bytes": cached * 2 * c["kv"] * c["dim"] * size + rows * (c["dim"] * 4 + 4),
                "flops": 4 * sum(n) * c["nodes"] * c["heads"] * c["dim"]}
    if c["op"] == "verify":
        rows = c["batch"] * c["nodes"]
        return {"bytes": rows * (c["vocab"] * (8 if c["sampled"] else 4) + 32), "flops": rows * c["vocab"] * (10 if c["sampled"] else 5)}
    row = 2 * c["layers"] * c["kv"] * c["dim"] * size
    if c["op"] == "compact":
        moved = sum(sum(1 for i, x in enumerate(p) if x != i) for p in _paths(c)[1])
        return {"bytes": 2 * moved * row + c["batch"] * (4 * c["nodes"] + 8), "flops": 0}
    return {"bytes": c["pages"] * (2 * c["page"] * row + 8), "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------
def _rows(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return dict(case, **globals()["_prepare_" + case["op"]](case, g, random.Random(int(seed))))


def _pools(c, g, pages, layers=1):
    """Keys and values of `layers` caches and their calibrated maxima (None: bf16)."""
    size = (layers, pages, c["page"], c["kv"], c["dim"])
    k, v = _rows(g, *size), _rows(g, *size)
    if c["cache"] == "bf16":
        return k.bfloat16(), v.bfloat16(), None, None
    amax = [torch.full((1,), a, device=DEV) for a in (4.0, 4.5)]
    k, v = ((x * (448.0 / a)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, a in zip((k, v), amax))
    return k, v, amax[0], amax[1]


def _prepare_append(c, g, r):
    t, heads, kv, dim = c["tokens"], c["heads"], c["kv"], c["dim"]
    kind = torch.float32 if c["src"] == "f32" else torch.bfloat16
    # the rows of one fused projection: q, k and v beside each other, a few channels far larger
    wide = torch.ones((heads + 2 * kv) * dim, device=DEV)
    wide[torch.randint(0, wide.numel(), (8,), device=DEV, generator=g)] = 12.0
    fused = (_rows(g, t, wide.numel()) * wide).to(kind)
    q, k, v = (x.view(t, -1, dim) for x in fused.split([heads * dim, kv * dim, kv * dim], dim=1))
    far = 65536
    where = torch.arange(t, device=DEV) + torch.randint(0, far - t, (1,), device=DEV, generator=g)
    angle = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * 1e6 ** (
        -torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
    pages = -(-t // c["page"]) + 3
    order = torch.randperm(pages, device=DEV, generator=g)
    at = torch.arange(t, device=DEV)
    slots = order[at // c["page"]] * c["page"] + at % c["page"]
    slots[t - c["pad"]:] = -1
    k_pool, v_pool, k_amax, v_amax = _pools(c, g, pages)
    return dict(q=q, k=k, v=v, positions=where, table=torch.cat([angle.cos(), angle.sin()], 1).float(), slots=slots,
                q_norm=1 + 0.2 * _rows(g, dim), k_norm=1 + 0.2 * _rows(g, dim), eps=1e-6, k_pool=k_pool[0], v_pool=v_pool[0],
                k_amax=k_amax, v_amax=v_amax, q_out=torch.zeros(t, heads, dim, device=DEV, dtype=torch.bfloat16))


def _block_table(c, g, lens, extra):
    each = [-(-n // c["page"]) for n in lens]
    order = torch.randperm(sum(each) + extra, device=DEV, generator=g).int()
    table = torch.zeros(len(lens), max(each), device=DEV, dtype=torch.int32)
    at = 0
    for b, e in enumerate(each):
        table[b, :e] = order[at:at + e]
        at += e
    return table, order.numel()


def _prepare_attend(c, g, r):
    n = _lengths(c["batch"], c["longest"], c["pad"])
    table, pages = _block_table(c, g, [x + c["nodes"] for x in n], 2)
    k, v, k_amax, v_amax = _pools(c, g, pages)
    trees = [_parents(r, c["nodes"], c["chain"]) for _ in n]
    for b in range(c["batch"] - c["pad"], c["batch"]):
        trees[b] = [-2] * c["nodes"]
    rows = c["batch"], c["nodes"], c["heads"]
    return dict(q=(2 * _rows(g, *rows, c["dim"])).bfloat16(), k_pool=k[0], v_pool=v[0], k_amax=k_amax, v_amax=v_amax,
                table=table, lens=torch.tensor(n, device=DEV, dtype=torch.int32), scale=c["dim"] ** -0.5,
                parents=torch.tensor(trees, device=DEV, dtype=torch.int32),
                out=torch.zeros(*rows, c["dim"], device=DEV, dtype=torch.bfloat16), lse=torch.zeros(*rows, device=DEV))


def _prepare_verify(c, g, r):
    b, w, n = c["batch"], c["nodes"], c["vocab"]
    trees = torch.tensor([_parents(r, w, c["sampled"]) for _ in range(b)], device=DEV, dtype=torch.int32)
    temperature = 0.6 + 0.6 * torch.rand(b, device=DEV, generator=g)
    temperature[:c["greedy"]] = 0
    logits, draft = 2.0 * _rows(g, b, w, n), None
    inner = trees.clamp_min(0).long()
    at = torch.arange(b, device=DEV)[:, None], inner
    if c["sampled"]:
        # the draft model is near the target: both have the same few likely tokens
        peaks = torch.randint(0, n, (b, w, 24), device=DEV, generator=g)
        logits.scatter_add_(2, peaks, 12 + 2 * _rows(g, b, w, 24))
        draft = logits + 0.5 * _rows(g, b, w, n)
        heat = torch.where(temperature > 0, temperature, 1.0)[:, None, None]
        chance = torch.rand(b, w, n, device=DEV, generator=g).clamp_min(1e-30)
        drawn = (draft / heat - torch.log(-torch.log(chance).clamp_min(1e-30))).argmax(-1)   # each row's own draw
        drafts = drawn[at]
    else:
        # a drafter's guesses: a node's children are among the likelier tokens after it
        drafts = torch.randint(0, n, (b, w), device=DEV, generator=g)
        logits.index_put_((*at, drafts), 12.5 + 1.5 * _rows(g, b, w), accumulate=True)
    return dict(logits=logits, draft=draft, drafts=drafts, parents=trees, temperature=temperature,
                uniforms=torch.rand(b, w + 1, device=DEV, generator=g),
                out=(torch.zeros(b, w, device=DEV, dtype=torch.int64), torch.zeros(b, w, device=DEV, dtype=torch.int32),
                     torch.zeros(b, device=DEV, dtype=torch.int32)))


def _paths(c):
    """The sizes' own accepted paths: the lengths of the sequences and the nodes each accepts."""
    r = random.Random(c["batch"] * 7919 + 5 * c["nodes"])
    paths = []
    for _ in range(c["batch"]):
        tree, path = _parents(r, c["nodes"], False), [0]
        for i in range(1, c["nodes"]):
            if tree[i] == path[-1] and r.random() < 0.6:
                path.append(i)
        paths.append(path)
    return _lengths(c["batch"], c["longest"]), paths


def _prepare_compact(c, g, r):
    n, paths = _paths(c)
    table, pages = _block_table(c, g, [x + c["nodes"] for x in n], 1)
    k, v, k_amax, v_amax = _pools(c, g, pages, c["layers"])
    padded = [p + [-1] * (c["nodes"] - len(p)) for p in paths]
    return dict(k_pool=k, v_pool=v, k_amax=k_amax, v_amax=v_amax, table=table, lens=torch.tensor(n, device=DEV, dtype=torch.int32),
                path=torch.tensor(padded, device=DEV, dtype=torch.int32),
                counts=torch.tensor([len(p) for p in paths], device=DEV, dtype=torch.int32))


def _prepare_copy(c, g, r):
    k, v, k_amax, v_amax = _pools(c, g, c["pool"], c["layers"])
    order = torch.randperm(c["pool"], device=DEV, generator=g).int()
    return dict(k_pool=k, v_pool=v, k_amax=k_amax, v_amax=v_amax, src=order[:c["pages"]].clone(),
                dst=order[c["pages"]:2 * c["pages"]].clone())


# ---- one pass ------------------------------------------------------------------------------------
def run(state):
    return globals()[("_own_" if own else "_plain_") + state["op"]](state)


def _kept(s):
    """The cache handles and the workspace that a serving program keeps beside its buffers."""
    import nvfp4_w4a4_block_act_amd as nv
    if "kept" not in s:
        caches = None
        if "k_pool" in s:
            pools = [(s["k_pool"], s["v_pool"])] if s["k_pool"].dim() == 4 else list(zip(s["k_pool"], s["v_pool"]))
            caches = [nv.PagedKVCache(k, v, s["k_amax"], s["v_amax"]) for k, v in pools]
        s["kept"] = caches, nv.Workspace(DEV)
    return (nv,) + s["kept"]


def _cache_values(s):
    kind = torch.float8_e4m3fn if s["cache"] == "fp8" else torch.bfloat16
    return {"k": s["k_pool"].view(kind), "v": s["v_pool"].view(kind)}


def _own_append(s):
    nv, caches, _ = _kept(s)
    nv.kv_append(s["k"], s["v"], caches[0], s["slots"], q=s["q"], positions=s["positions"], rope=s["table"],
                 interleaved=s["inter"], q_out=s["q_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"])
    return dict(_cache_values(s), q=s["q_out"])


def _own_attend(s):
    nv, caches, ws = _kept(s)
    out, lse = nv.attn_tree(s["q"], caches[0], s["table"], s["lens"], parents=s["parents"], max_len=s["longest"],
                            scale=s["scale"], window=s["window"], workspace=ws, out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def _own_verify(s):
    nv, _, ws = _kept(s)
    tokens, path, counts = nv.verify_drafts(s["logits"], s["drafts"], s["parents"], s["temperature"], s["uniforms"],
                                            draft_logits=s["draft"], workspace=ws, out=s["out"])
    return {"tokens": tokens, "path": path, "counts": counts}


def _own_compact(s):
    nv, caches, _ = _kept(s)
    nv.kv_compact(s["table"], s["lens"], s["path"], s["counts"], caches)
    return _cache_values(s)


def _own_copy(s):
    nv, caches, _ = _kept(s)
    nv.kv_copy_pages(s["src"], s["dst"], caches)
    return _cache_values(s)


# ---- plain forms ---------------------------------------------------------------------------------
def _rotated(x, cos, sin, rot, inter):
    head = x[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., : rot // 2], head[..., rot // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _coded(x, amax):
    """bf16 values in the cache's type: E4M3 codes of x * fl(448 / amax), or themselves."""
    if amax is None:
        return x
    gain = torch.full_like(amax, 448.0) / amax      # a quotient of tensors: rounded once
    return (x.float() * gain).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    n = s["tokens"] - s["pad"]  # padded rows come last
    turn = s["table"][s["positions"][:n]][:, None, :]
    cos, sin = turn[..., : s["rot"] // 2], turn[..., s["rot"] // 2:]
    q, k = s["q"][:n].float(), s["k"][:n].float()
    q, k = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w for x, w in ((q, s["q_norm"]), (k, s["k_norm"])))
    s["q_out"][:n] = _rotated(q, cos, sin, s["rot"], s["inter"]).bfloat16()
    k = _rotated(k, cos, sin, s["rot"], s["inter"]).bfloat16()
    s["k_pool"].flatten(0, 1)[s["slots"][:n]] = _coded(k, s["k_amax"])
    s["v_pool"].flatten(0, 1)[s["slots"][:n]] = _coded(s["v"][:n].bfloat16(), s["v_amax"])
    return dict(_cache_values(s), q=s["q_out"])


def _values(pool, amax):
    return pool.float() if amax is None else pool.view(torch.float8_e4m3fn).float() * (amax / 448.0)


def _ancestors(parents):
    """[b, i, j]: whether node i has node j on its way up, itself included; no j at all for a padded node."""
    b, w = parents.shape
    anc = torch.zeros(b, w, w, device=DEV, dtype=torch.bool)
    for i in range(w):
        up = parents[:, i].long()
        if i > 0:
            at = up.clamp(0, i - 1)
            above = anc.gather(1, at[:, None, None].expand(b, 1, w))[:, 0]
            anc[:, i] = above & (up >= 0)[:, None]
            fine = (up == -1) | ((up >= 0) & (up < i) & above.gather(1, at[:, None])[:, 0])
        else:
            fine = up == -1
        anc[:, i, i] = fine
        anc[:, i] &= fine[:, None]
    return anc


def _plain_attend(s):
    b, w, h, kv, d = s["batch"], s["nodes"], s["heads"], s["kv"], s["dim"]
    n, many = s["longest"] + w, h // kv
    pages = s["table"].shape[1]
    table, at = s["table"].long(), torch.arange(min(n, pages * s["page"]), device=DEV)
    k, v = (_values(s[x + "_pool"][table].flatten(1, 2)[:, :n], s[x + "_amax"]) for x in "kv")  # b, n, kv, d
    lens, anc = s["lens"].long()[:, None, None], _ancestors(s["parents"])
    far = at - lens                                                                             # b, 1, n: which drafted token
    drafted = (far >= 0) & (far < w)
    seen = torch.where(drafted, anc.gather(2, far.clamp(0, w - 1).expand(b, w, -1)), (far < 0) & anc.any(-1, keepdim=True))
    if s["window"]:
        later = seen.flip(-1).cumsum(-1).flip(-1)                                               # seen from here to the end
        seen &= later <= s["window"]
    q = s["q"].float().view(b, w, kv, many, d).permute(0, 2, 1, 3, 4).reshape(b, kv, w * many, d)
    logits = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(b, kv, w, many, -1) * s["scale"]
    logits = logits.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top.clamp_min(-1e30))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, kv, w * many, -1), v.permute(0, 2, 1, 3).contiguous()).view(b, kv, w, many, d)
    out = (out / total.clamp_min(1e-30)).permute(0, 2, 1, 3, 4).reshape(b, w, h, d)
    lse = (top + torch.log(total)).permute(0, 2, 1, 3, 4).reshape(b, w, h)
    return {"out": out.bfloat16(), "lse": lse}


def _softmax(x, heat):
    """In 64 bits: the running sums of many small weights are compared with one number."""
    x = x.double() / heat.double()[:, None, None]
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return x / x.sum(-1, keepdim=True)


def _plain_verify(s):
    b, w, n = s["batch"], s["nodes"], s["vocab"]
    row = torch.arange(b, device=DEV)
    greedy = ~(s["temperature"] > 0)
    heat = torch.where(greedy, 1.0, s["temperature"])
    largest = s["logits"].argmax(-1)
    p = _softmax(s["logits"], heat)
    q = _softmax(s["draft"], heat) if s["sampled"] else None
    up, drafts, u = s["parents"].long(), s["drafts"], s["uniforms"].double()
    now, count, sum_ = torch.zeros(b, device=DEV, dtype=torch.int64), torch.ones(b, device=DEV, dtype=torch.int64), u.new_zeros(b)
    tried = torch.zeros(b, w, device=DEV, dtype=torch.bool)                  # children of the node reached, and turned down
    tokens, path = torch.full((b, w), -1, device=DEV), torch.full((b, w), -1, device=DEV)
    path[:, 0] = 0
    for i in range(1, w):
        x, child = drafts[:, i], up[:, i] == now
        new = child & ~(tried & (drafts == x[:, None])).any(-1)
        if s["sampled"]:
            new = child & ~tried.any(-1)
            chosen = u[row, now] * q[row, now, x] < p[row, now, x]
        else:
            sum_ = torch.where(new, sum_ + p[row, now, x], sum_)
            chosen = u[row, now] < sum_
        take = torch.where(greedy, child & (x == largest[row, now]), new & chosen)
        tried[:, i] = child
        tried &= ~take[:, None]
        now, sum_ = torch.where(take, i, now), torch.where(take, 0.0, sum_)
        tokens[row, count - 1] = torch.where(take, x, tokens[row, count - 1])
        path[row, count.clamp_max(w - 1)] = torch.where(take, i, path[row, count.clamp_max(w - 1)])
        count += take
    rest = p[row, now]
    if s["sampled"]:
        rest = torch.where(tried.any(-1, keepdim=True), (rest - q[row, now]).clamp_min(0), rest)
    else:
        gone = torch.zeros(b, n, device=DEV, dtype=torch.int32).scatter_add_(1, drafts, tried.int())
        rest = torch.where(gone > 0, 0.0, rest)
    run_ = rest.cumsum(-1)
    last = (run_ <= u[:, w:] * run_[:, -1:]).sum(-1).clamp_max(n - 1)
    tokens[row, count - 1] = torch.where(greedy, largest[row, now], last)
    return {"tokens": tokens, "path": path.int(), "counts": count.int()}


def _plain_compact(s):
    w = s["nodes"]
    i = torch.arange(w, device=DEV)
    start, moved = s["lens"].long()[:, None], (i < s["counts"][:, None]) & (s["path"] >= 0)

    def row(at):
        return s["table"].long().gather(1, at // s["page"]) * s["page"] + at % s["page"]
    frm, to = row(start + s["path"].clamp_min(0).long()), row(start + i)
    to = torch.where(moved, to, frm)                                     # a row that stays is written onto itself
    keep = moved | ~(frm[:, :, None] == torch.where(moved, to, -1)[:, None, :]).any(-1)
    frm, to = frm[keep], to[keep]
    for pool in (s["k_pool"], s["v_pool"]):
        rows = pool.flatten(1, 2)
        rows[:, to] = rows[:, frm]
    return _cache_values(s)


def _plain_copy(s):
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, s["dst"].long()] = pool[:, s["src"].long()]
    return _cache_values(s)


# ---- 64 bits, from the definitions ---------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _pool_values(pool, cache):
    return (pool.view(torch.float8_e4m3fn) if cache == "fp8" else pool).double()


def _exact_head(x, w, s):
    """The norm, then a complex rotation of the pairs of the first `rot` elements, one complex number a pair."""
    x = x.double()
    x = w.double() * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt()
    r, half = s["rot"], s["rot"] // 2
    turn = s["table"][s["positions"]].double()
    z = torch.complex(turn[:, :half], turn[:, half:])[:, None, :]
    pair = x[..., :r].unflatten(-1, (half, 2)) if s["inter"] else x[..., :r].unflatten(-1, (2, half)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    x[..., :r] = y.flatten(-2) if s["inter"] else y.transpose(-1, -2).flatten(-2)
    return x


def _nearest_e4m3(y):
    """Nearest E4M3 value, ties to even, of |y| <= 448: steps of 2^(e - 3), at least 2^-9."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_append(s):
    ok = torch.nonzero(s["slots"] >= 0).flatten()
    got = {"q": s["q_out"].double()}
    got["q"][ok] = _exact_head(s["q"], s["q_norm"], s)[ok]
    for x in "kv":
        rows = (_exact_head(s["k"], s["k_norm"], s) if x == "k" else s["v"].double())[ok]
        amax = s[x + "_amax"]
        if amax is not None:  # by definition a code is that of the bf16 value times fl(448 / amax), a product in 32 bits
            gain = torch.full_like(amax, 448.0) / amax
            rows = _nearest_e4m3((rows.bfloat16().float() * gain).double().clamp(-448, 448))
        pool = _pool_values(s[x + "_pool"], s["cache"])
        pool.view(-1, s["kv"], s["dim"])[s["slots"][ok]] = rows
        got[x] = pool
    return got


def _way_up(tree, i):
    """The nodes from node i to the context, itself first; none if the way leads nowhere."""
    way = []
    while 0 <= i:
        way.append(i)
        if not -1 <= tree[i] < i:
            return []
        i = tree[i]
    return way


def _exact_attend(s):
    b, w, h, kv, d = s["batch"], s["nodes"], s["heads"], s["kv"], s["dim"]
    out = torch.zeros(b, w, h, d, device=DEV, dtype=torch.float64)
    lse = torch.full((b, w, h), -math.inf, device=DEV, dtype=torch.float64)
    trees = s["parents"].tolist()
    for x, n in enumerate(_lengths(b, s["longest"], s["pad"])):
        mask = torch.zeros(w, n + w, dtype=torch.bool)
        for i in range(w):
            way = _way_up(trees[x], i)
            if way:
                cols = list(range(n)) + sorted(n + j for j in way)
                cols = cols[-s["window"]:] if s["window"] else cols
                mask[i, cols] = True
        if not mask.any():
            continue
        mask = mask.to(DEV)
        at = torch.arange(n + w, device=DEV)
        page, inside = s["table"][x].long()[at // s["page"]], at % s["page"]
        for y in range(kv):
            k, v = (_pool_values(s[z + "_pool"][page, inside, y], s["cache"]) for z in "kv")
            if s["cache"] == "fp8":
                k, v = k * (s["k_amax"].double() / 448), v * (s["v_amax"].double() / 448)
            heads = slice(y * (h // kv), (y + 1) * (h // kv))
            q = s["q"][x, :, heads].double().flatten(0, 1)
            score = s["scale"] * torch.mm(q, k.t().contiguous())
            score[~mask.repeat_interleave(h // kv, 0)] = -math.inf
            total = torch.logsumexp(score, -1)
            p = torch.nan_to_num(torch.exp(score - total[:, None]))
            out[x, :, heads] = torch.mm(p, v).view(w, -1, d)
            lse[x, :, heads] = total.view(w, -1)
    return {"out": out, "lse": lse}


def _exact_verify(s):
    b, w = s["batch"], s["nodes"]
    tokens, path, counts = [], [], []
    trees, drafts, u, heat = (s[x].tolist() for x in ("parents", "drafts", "uniforms", "temperature"))
    for x in range(b):
        node, said, way = 0, [], [0]
        while True:
            row = s["logits"][x, node].double()
            kids = [c for c in range(node + 1, w) if trees[x][c] == node]
            taken = None
            if heat[x] == 0:
                best = int(row.argmax())
                taken = next((c for c in kids if drafts[x][c] == best), None)
            else:
                p = torch.softmax(row / heat[x], 0)
                if s["sampled"]:
                    if kids:
                        q, t = torch.softmax(s["draft"][x, node].double() / heat[x], 0), drafts[x][kids[0]]
                        if u[x][node] * float(q[t]) < float(p[t]):
                            taken = kids[0]
                        else:
                            p = torch.relu(p - q)
                else:
                    mass, seen = 0.0, set()
                    for c in kids:
                        if drafts[x][c] not in seen:
                            seen.add(drafts[x][c])
                            mass += float(p[drafts[x][c]])
                            if u[x][node] < mass:
                                taken = c
                                break
                    else:
                        p[list(seen)] = 0.0
            if taken is None:
                break
            node = taken
            way.append(node)
            said.append(drafts[x][node])
        if heat[x] > 0:
            total = torch.cumsum(p, 0)
            best = min(int(torch.searchsorted(total, u[x][w] * total[-1:], right=True)[0]), s["vocab"] - 1)
        said.append(best)
        tokens.append(said + [-1] * (w - len(said)))
        path.append(way + [-1] * (w - len(way)))
        counts.append(len(way))
    kinds = zip((tokens, path, counts), (torch.int64, torch.int32, torch.int32))
    return dict(zip(("tokens", "path", "counts"), (torch.tensor(x, device=DEV, dtype=k) for x, k in kinds)))


def _exact_compact(s):
    n, paths = _paths(s)
    table, page = s["table"].tolist(), s["page"]
    frm, to = [], []
    for x, way in enumerate(paths):
        for i, j in enumerate(way):
            if i != j:
                for where, at in ((frm, n[x] + j), (to, n[x] + i)):
                    where.append(table[x][at // page] * page + at % page)
    frm, to = (torch.tensor(x, device=DEV, dtype=torch.int64) for x in (frm, to))
    got = {}
    for x in "kv":
        old = _pool_values(s[x + "_pool"], s["cache"])
        got[x] = old.clone()
        got[x].flatten(1, 2)[:, to] = old.flatten(1, 2)[:, frm]
    return got


def _exact_copy(s):
    got = {}
    for x in "kv":
        got[x] = _pool_values(s[x + "_pool"], s["cache"])
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            got[x][:, b] = _pool_values(s[x + "_pool"][:, a], s["cache"])
    return got
