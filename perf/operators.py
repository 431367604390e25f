"""The token mixers of a served hybrid model, as workloads: appending to a paged key-value cache,
attention of one new token over it, and the gated linear attention of the recurrent layers in its
single-token and its prompt form.

Each workload has a plain form in elementary torch operations and the call of the library that does
the same work; `own` says which of the two `run` takes.  Head counts and sizes are those of this
repository's workloads where it has them (8 key-value heads of 128 beside 5120 channels, a 32768-token
cache of 1024 channels, a recurrent layer of 16 query/key and 32 value heads of 128).

Definitions (the plain forms below are their direct transcription):

  append   The first `rot` elements of each head of q and k are rotated by the angle of the token's
           position (fp32 tables of cos and sin; pairs (i, i + rot/2), or (2i, 2i + 1) interleaved),
           rounded to bf16, and k and v go to the cache row `slot`: as bf16, or as E4M3 codes of
           x * (448 / amax).  A negative slot marks a padded row, of which nothing is written.
  attend   out[b, h] = sum_j softmax_j(scale * q[b, h] . K_j) V_j over the last `window` of the
           first len[b] cached tokens (all of them if window == 0), and the softmax's log sum;
           zeros and -inf where there is no token.
  gdn      S_t = e^{g_t} S_{t-1} + beta_t k_t (v_t - (e^{g_t} S_{t-1})^T k_t)^T,  o_t = scale S_t^T q_t;
           without beta: S_t = e^{g_t} S_{t-1} + k_t v_t^T (linear attention with a decay for each head).
"""
import math
import random

import torch

own = False
DEV = "cuda:0"
CHUNK = 64          # tokens of a chunk in the plain chunked form


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    """Smallest, ordinary and largest call of each operator."""
    append = dict(op="append", heads=40, kv=8, dim=128, rot=128, inter=False, page=64, pad=0)
    attend = dict(op="attend", heads=40, kv=8, dim=128, page=64, window=0)
    step = dict(op="step", kheads=16, vheads=32, dim=128, vdim=128, delta=True)
    prompt = dict(op="prompt", kheads=16, vheads=32, dim=128, vdim=128, delta=True, warm=False)
    return [
        # one request decoding: the rows of the fused fp32 projection go to an FP8 cache
        dict(append, name="append_1_f32_fp8", tokens=1, src="f32", cache="fp8"),
        # a decoding batch padded to its captured size, half of each head rotated, bf16 cache
        dict(append, name="append_133_bf16_bf16", tokens=133, pad=5, src="bf16", cache="bf16", rot=64, inter=True, page=16),
        # a whole 32768-token prompt of the 8 x 128 cache
        dict(append, name="append_32768_f32_fp8", tokens=32768, src="f32", cache="fp8"),
        # one chat turn of one request: latency
        dict(attend, name="attend_1x517_fp8", batch=1, longest=517, cache="fp8", pad=0),
        # an ordinary serving batch of uneven lengths, padded by three rows
        dict(attend, name="attend_67x4099_fp8", batch=67, longest=4099, cache="fp8", pad=3),
        # few long documents over wide heads, bf16 cache
        dict(attend, name="attend_6x32768_bf16", batch=6, longest=32768, cache="bf16", pad=0, heads=24, kv=4, dim=256, page=128),
        # one token through one recurrent layer for one request, a batch, and a full batch
        dict(step, name="step_1", batch=1, pad=0),
        dict(step, name="step_61", batch=61, pad=3),
        dict(step, name="step_256", batch=256, pad=0),
        # uneven short prompts in one call
        dict(prompt, name="prompt_5x300", batch=5, longest=300, warm=True),
        # one 8192-token prompt
        dict(prompt, name="prompt_1x8192", batch=1, longest=8192),
        # a prefill batch at a 32768-token budget, plain linear attention with a decay
        dict(prompt, name="prompt_6x8192_linear", batch=6, longest=8192, delta=False, warm=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case: sizes spread over their logarithm, the operators in turn by chance."""
    op = rng.choice(["append", "attend", "step", "prompt"])
    if op == "append":
        heads, kv, dim = rng.choice([(40, 8, 128), (32, 8, 128), (24, 4, 256), (16, 16, 64), (16, 1, 128)])
        tokens = _log(rng, 1, 24000)
        return dict(op=op, heads=heads, kv=kv, dim=dim, rot=rng.choice([dim, dim // 2, 32]), inter=rng.random() < 0.3,
                    page=rng.choice([16, 48, 64, 128]), pad=rng.choice([0, 0, min(tokens - 1, 7)]), tokens=tokens,
                    src=rng.choice(["f32", "bf16"]), cache=rng.choice(["fp8", "bf16"]))
    if op == "attend":
        heads, kv, dim = rng.choice([(40, 8, 128), (32, 8, 128), (24, 4, 256), (16, 16, 64), (48, 2, 128)])
        batch = _log(rng, 1, 160)
        longest = _log(rng, 16, min(32768, 196608 * 1024 // (batch * kv * dim)))
        return dict(op=op, heads=heads, kv=kv, dim=dim, page=rng.choice([16, 48, 64, 128]),
                    window=rng.choice([0, 0, max(1, longest // 3)]), batch=batch, longest=longest,
                    cache=rng.choice(["fp8", "bf16"]), pad=rng.choice([0, min(batch - 1, 3)]))
    kheads, vheads, dim, vdim = rng.choice([(16, 32, 128, 128), (8, 32, 128, 128), (16, 16, 64, 128), (4, 4, 128, 256)])
    if op == "step":
        batch = _log(rng, 1, 200)
        return dict(op=op, kheads=kheads, vheads=vheads, dim=dim, vdim=vdim, delta=rng.random() < 0.7, batch=batch,
                    pad=rng.choice([0, min(batch - 1, 3)]))
    batch = _log(rng, 1, 12)
    return dict(op=op, kheads=kheads, vheads=vheads, dim=dim, vdim=vdim, delta=rng.random() < 0.7, batch=batch,
                longest=_log(rng, 1, 32768 // batch), warm=rng.random() < 0.5)


def _lengths(batch, longest, pad=0):
    """Uneven lengths of a batch, one of them the longest; `pad` empty rows at its end."""
    r = random.Random(batch * 1000003 + longest)
    n = [r.randint(max(1, longest // 4), longest) for _ in range(batch)]
    n[r.randrange(batch - pad)] = longest
    return n[: batch - pad] + [0] * pad if pad else n


def _attended(c):
    return [min(n, c["window"]) if c["window"] else n for n in _lengths(c["batch"], c["longest"], c["pad"])]


def work(case):
    c = case
    if c["op"] == "append":
        t, src, dst = c["tokens"] - c["pad"], 4 if c["src"] == "f32" else 2, 1 if c["cache"] == "fp8" else 2
        q, kv = c["heads"] * c["dim"], 2 * c["kv"] * c["dim"]
        table = 4 * c["rot"] + 16
        return {"bytes": t * ((q + kv) * src + 2 * q + kv * dst + table), "flops": 3 * t * c["rot"] * (c["heads"] + c["kv"])}
    if c["op"] == "attend":
        n, size = sum(_attended(c)), 1 if c["cache"] == "fp8" else 2
        rows = c["batch"] * c["heads"]
        return {"bytes": n * 2 * c["kv"] * c["dim"] * size + rows * (c["dim"] * 4 + 4), "flops": 4 * n * c["heads"] * c["dim"]}
    state = c["vheads"] * c["dim"] * c["vdim"]
    token = 2 * (2 * c["kheads"] * c["dim"] + 2 * c["vheads"] * c["vdim"]) + 4 * c["vheads"] * (2 if c["delta"] else 1)
    once = (7 if c["delta"] else 5) * state  # decay, k S, update, q S for one token
    if c["op"] == "step":
        b = c["batch"] - c["pad"]
        return {"bytes": b * (8 * state + token), "flops": b * once}
    t = sum(_lengths(c["batch"], c["longest"]))
    return {"bytes": t * token + 4 * c["batch"] * state * (2 if c["warm"] else 1), "flops": t * once}


# ---- inputs --------------------------------------------------------------------------------------
def _rows(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return dict(case, **globals()["_prepare_" + case["op"]](case, g))


def _prepare_append(c, g):
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
    size = (pages, c["page"], kv, dim)
    if c["cache"] == "fp8":
        pool = [torch.randint(0, 0x7E, size, device=DEV, generator=g, dtype=torch.uint8) for _ in range(2)]
        amax = [torch.full((1,), a, device=DEV) for a in (4.5, 6.0)]
    else:
        pool, amax = [_rows(g, *size).bfloat16() for _ in range(2)], [None, None]
    return dict(q=q, k=k, v=v, positions=where, table=torch.cat([angle.cos(), angle.sin()], 1).float(), slots=slots,
                k_pool=pool[0], v_pool=pool[1], k_amax=amax[0], v_amax=amax[1],
                q_out=torch.zeros(t, heads, dim, device=DEV, dtype=torch.bfloat16))


def _prepare_attend(c, g):
    n = _lengths(c["batch"], c["longest"], c["pad"])
    each = [-(-x // c["page"]) for x in n]
    pages = sum(each) + 2
    order = torch.randperm(pages, device=DEV, generator=g).int()
    table = torch.zeros(c["batch"], max(each), device=DEV, dtype=torch.int32)
    at = 0
    for b, e in enumerate(each):
        table[b, :e] = order[at:at + e]
        at += e
    size = (pages, c["page"], c["kv"], c["dim"])
    k, v = _rows(g, *size), _rows(g, *size)
    amax = [None, None]
    if c["cache"] == "fp8":
        amax = [torch.full((1,), a, device=DEV) for a in (4.0, 4.5)]
        k, v = ((x * (448.0 / a)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, a in zip((k, v), amax))
    else:
        k, v = k.bfloat16(), v.bfloat16()
    rows = c["batch"], c["heads"]
    return dict(q=(2 * _rows(g, *rows, c["dim"])).bfloat16(), k_pool=k, v_pool=v, k_amax=amax[0], v_amax=amax[1],
                table=table, lens=torch.tensor(n, device=DEV, dtype=torch.int32), scale=c["dim"] ** -0.5,
                out=torch.zeros(*rows, c["dim"], device=DEV, dtype=torch.bfloat16), lse=torch.zeros(*rows, device=DEV))


def _prepare_mixer(c, g, t, states):
    """Queries and keys of unit length, gates as the recurrent layers make them: e^-(A * softplus(dt))."""
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1).bfloat16()  # noqa: E731
    hv = c["vheads"]
    rate = 1 + 15 * torch.rand(hv, device=DEV, generator=g)
    dt = torch.exp(math.log(1e-3) + (math.log(0.1) - math.log(1e-3)) * torch.rand(t, hv, device=DEV, generator=g))
    state = 0.5 * _rows(g, states, hv, c["dim"], c["vdim"])
    return dict(q=unit(_rows(g, t, c["kheads"], c["dim"])), k=unit(_rows(g, t, c["kheads"], c["dim"])),
                v=_rows(g, t, hv, c["vdim"]).bfloat16(), g=-rate * dt,
                beta=torch.sigmoid(_rows(g, t, hv)) if c["delta"] else None, state=state, scale=c["dim"] ** -0.5,
                out=torch.zeros(t, hv, c["vdim"], device=DEV, dtype=torch.bfloat16))


def _prepare_step(c, g):
    s = _prepare_mixer(c, g, c["batch"], c["batch"] + 2)
    index = torch.randperm(c["batch"] + 2, device=DEV, generator=g)[: c["batch"]].int()
    index[c["batch"] - c["pad"]:] = -1
    return dict(s, index=index)


def _prepare_prompt(c, g):
    n = _lengths(c["batch"], c["longest"])
    s = _prepare_mixer(c, g, sum(n), c["batch"] + 1)
    ends = torch.tensor([0] + n, device=DEV).cumsum(0).int()
    index = torch.randperm(c["batch"] + 1, device=DEV, generator=g)[: c["batch"]].int()
    has = torch.ones(c["batch"], device=DEV, dtype=torch.int32) if c["warm"] else None
    return dict(s, ends=ends, index=index, has=has)


# ---- one pass ------------------------------------------------------------------------------------
def run(state):
    return globals()[("_own_" if own else "_plain_") + state["op"]](state)


def _kept(s):
    """The cache handle and the workspace that a serving program keeps beside its buffers."""
    import nvfp4_w4a4_block_act_amd as nv
    if "kept" not in s:
        s["kept"] = nv.PagedKVCache(s["k_pool"], s["v_pool"], s["k_amax"], s["v_amax"]) if "k_pool" in s else None, nv.Workspace(DEV)
    return (nv,) + s["kept"]


def _cache_values(s):
    kind = torch.float8_e4m3fn if s["cache"] == "fp8" else torch.bfloat16
    return {"q": s["q_out"], "k": s["k_pool"].view(kind), "v": s["v_pool"].view(kind)}


def _own_append(s):
    nv, cache, _ = _kept(s)
    nv.kv_append(s["k"], s["v"], cache, s["slots"], q=s["q"], positions=s["positions"], rope=s["table"],
                 interleaved=s["inter"], q_out=s["q_out"])
    return _cache_values(s)


def _own_attend(s):
    nv, cache, ws = _kept(s)
    out, lse = nv.attn_decode(s["q"], cache, s["table"], s["lens"], max_len=s["longest"], scale=s["scale"],
                              window=s["window"], workspace=ws, out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def _own_step(s):
    nv, _, _ = _kept(s)
    nv.gdn_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], state_index=s["index"], scale=s["scale"], out=s["out"])
    return {"out": s["out"], "state": s["state"]}


def _own_prompt(s):
    nv, _, ws = _kept(s)
    nv.gdn_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["ends"], has_state=s["has"],
                   state_index=s["index"], scale=s["scale"], workspace=ws, out=s["out"])
    return {"out": s["out"], "state": s["state"]}


# ---- plain forms ---------------------------------------------------------------------------------
def _rotated(x, cos, sin, rot, inter):
    head = x[..., :rot]
    a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., : rot // 2], head[..., rot // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _coded(x, amax):
    """bf16 values in the cache's type: E4M3 codes of x * (448 / amax), or themselves."""
    if amax is None:
        return x
    return (x.float() * (448.0 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    n = s["tokens"] - s["pad"]  # padded rows come last
    turn = s["table"][s["positions"][:n]][:, None, :]
    cos, sin = turn[..., : s["rot"] // 2], turn[..., s["rot"] // 2:]
    s["q_out"][:n] = _rotated(s["q"][:n].float(), cos, sin, s["rot"], s["inter"]).bfloat16()
    k = _rotated(s["k"][:n].float(), cos, sin, s["rot"], s["inter"]).bfloat16()
    s["k_pool"].flatten(0, 1)[s["slots"][:n]] = _coded(k, s["k_amax"])
    s["v_pool"].flatten(0, 1)[s["slots"][:n]] = _coded(s["v"][:n].bfloat16(), s["v_amax"])
    return _cache_values(s)


def _values(pool, amax):
    return pool.float() if amax is None else pool.view(torch.float8_e4m3fn).float() * (amax / 448.0)


def _plain_attend(s):
    b, h, kv, d, n = s["batch"], s["heads"], s["kv"], s["dim"], s["longest"]
    table = s["table"].long()
    k, v = (_values(s[x + "_pool"][table].flatten(1, 2)[:, :n], s[x + "_amax"]) for x in "kv")  # b, n, kv, d
    at = torch.arange(n, device=DEV)
    lens = s["lens"].long()[:, None]
    low = (lens - s["window"]).clamp_min(0) if s["window"] else torch.zeros_like(lens)
    seen = ((at >= low) & (at < lens))[:, None, None, :]
    q = s["q"].float().view(b, kv, h // kv, d)
    logits = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * s["scale"]
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top.clamp_min(-1e30))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous()) / total.clamp_min(1e-30)
    return {"out": out.view(b, h, d).bfloat16(), "lse": (top + torch.log(total)).view(b, h)}


def _plain_step(s):
    n = s["batch"] - s["pad"]  # padded rows come last
    hv, many = s["vheads"], s["vheads"] // s["kheads"]
    q, k = (s[x][:n].float().repeat_interleave(many, 1) for x in "qk")
    v, at = s["v"][:n].float(), s["index"][:n].long()
    S = s["state"][at] * torch.exp(s["g"][:n])[..., None, None]
    if s["delta"]:
        v = s["beta"][:n, :, None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * v[..., None, :]
    s["out"][:n] = (s["scale"] * (S * q[..., None]).sum(-2)).bfloat16()
    s["state"][at] = S
    return {"out": s["out"], "state": s["state"]}


def _padded(x, s, many=1):
    """Rows of all sequences -> [sequence, head, chunk, row, ...] in fp32, zeros behind each sequence's end."""
    n = s["ends"].long()
    longest = -(-s["longest"] // CHUNK) * CHUNK
    at = torch.arange(longest, device=DEV)
    inside = at < (n[1:] - n[:-1])[:, None]
    rows = x.float()[torch.where(inside, n[:-1, None] + at, 0)]
    rows = torch.where(inside.view(*inside.shape, *[1] * (x.dim() - 1)), rows, 0.0)
    return rows.repeat_interleave(many, 2).transpose(1, 2).unflatten(2, (-1, CHUNK)).contiguous(), inside


def _plain_prompt(s):
    """Chunks of 64 tokens: products within a chunk at once, the state from chunk to chunk."""
    many = s["vheads"] // s["kheads"]
    (q, inside), (k, _), (v, _), (g, _) = _padded(s["q"], s, many), _padded(s["k"], s, many), _padded(s["v"], s), _padded(s["g"], s)
    past = g.double().cumsum(-1)                                   # log of the decay since the chunk's start
    low = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    fade = torch.exp((past[..., :, None] - past[..., None, :]).masked_fill(~low, -math.inf)).float()
    since, left = torch.exp(past).float()[..., None], torch.exp(past[..., -1:] - past).float()[..., None]
    kt = k.transpose(-1, -2).contiguous()
    scores = torch.matmul(q, kt) * fade
    if s["delta"]:
        beta = _padded(s["beta"], s)[0][..., None]
        A = beta * torch.matmul(k, kt) * fade
        solve = torch.eye(CHUNK, device=DEV).expand_as(A).clone()  # (1 + strictly lower A)^-1, row by row
        for i in range(1, CHUNK):
            solve[..., i, :i] = -(A[..., i, :i, None] * solve[..., :i, :i]).sum(-2)
    at = s["index"].long()
    S = s["state"][at] if s["warm"] else torch.zeros_like(s["state"][at])
    out = []
    for c in range(q.shape[2]):
        new = v[:, :, c]
        if s["delta"]:
            new = torch.matmul(solve[:, :, c], beta[:, :, c] * (new - since[:, :, c] * torch.matmul(k[:, :, c], S)))
        out.append(since[:, :, c] * torch.matmul(q[:, :, c], S) + torch.matmul(scores[:, :, c], new))
        S = since[:, :, c, -1:] * S + torch.matmul(kt[:, :, c], left[:, :, c] * new)
    o = (s["scale"] * torch.stack(out, 2)).flatten(2, 3).transpose(1, 2)
    row = torch.arange(s["q"].shape[0], device=DEV)
    which = torch.searchsorted(s["ends"][1:].long(), row, right=True)
    s["out"].copy_(o[which, row - s["ends"].long()[which]])
    s["state"][at] = S
    return {"out": s["out"], "state": s["state"]}


# ---- 64 bits, from the definitions ---------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)


def _exact_turn(x, s):
    """Complex rotation of the pairs of the first `rot` elements, one complex number a pair."""
    x = x.double()
    r, half = s["rot"], s["rot"] // 2
    turn = s["table"][s["positions"]].double()
    z = torch.complex(turn[:, :half], turn[:, half:])[:, None, :]
    pair = x[..., :r].unflatten(-1, (half, 2)) if s["inter"] else x[..., :r].unflatten(-1, (2, half)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    y = x.clone()
    y[..., :r] = w.flatten(-2) if s["inter"] else w.transpose(-1, -2).flatten(-2)
    return y


def _nearest_e4m3(y):
    """Nearest E4M3 value, ties to even, of |y| <= 448: steps of 2^(e - 3), at least 2^-9."""
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_append(s):
    ok = torch.nonzero(s["slots"] >= 0).flatten()
    got = {"q": s["q_out"].double(), "k": None, "v": None}
    got["q"][ok] = _exact_turn(s["q"], s)[ok]
    for x in "kv":
        rows = (_exact_turn(s["k"], s) if x == "k" else s["v"].double())[ok]
        amax = s[x + "_amax"]
        if amax is not None:  # by definition a code is that of the bf16 value times 448 / amax, a product in 32 bits
            rows = _nearest_e4m3((rows.bfloat16().float() * (448.0 / amax)).double().clamp(-448, 448))
            pool = s[x + "_pool"].view(torch.float8_e4m3fn).double()
        else:
            pool = s[x + "_pool"].double()
        pool.view(-1, s["kv"], s["dim"])[s["slots"][ok]] = rows
        got[x] = pool
    return got


def _exact_attend(s):
    b, h, kv, d = s["batch"], s["heads"], s["kv"], s["dim"]
    out, lse = torch.zeros(b, h, d, device=DEV, dtype=torch.float64), torch.full((b, h), -math.inf, device=DEV, dtype=torch.float64)
    for i, n in enumerate(_lengths(b, s["longest"], s["pad"])):
        first = max(0, n - s["window"]) if s["window"] else 0
        if n == first:
            continue
        at = torch.arange(first, n, device=DEV)
        page, inside = s["table"][i].long()[at // s["page"]], at % s["page"]
        k, v = s["k_pool"][page, inside], s["v_pool"][page, inside]
        if s["cache"] == "fp8":
            k, v = (x.view(torch.float8_e4m3fn).double() * (s[y].double() / 448) for x, y in ((k, "k_amax"), (v, "v_amax")))
        k, v = (x.double().transpose(0, 1).repeat_interleave(h // kv, 0) for x in (k, v))   # h, n, d
        logit = s["scale"] * (k * s["q"][i].double()[:, None, :]).sum(-1)
        lse[i] = torch.logsumexp(logit, -1)
        out[i] = (torch.exp(logit - lse[i][:, None])[..., None] * v).sum(1)
    return {"out": out, "lse": lse}


def _exact_recurrence(s, rows):
    """Token by token; rows[t]: the rows of the sequences that have a t-th token, the longest ones first."""
    many = s["vheads"] // s["kheads"]
    q, k = (s[x].double().repeat_interleave(many, 1) for x in "qk")
    v, g, out = s["v"].double(), s["g"].double(), s["out"].double()
    beta = s["beta"].double() if s["delta"] else None
    S = s["first"]
    for r in rows:
        n = r.numel()
        now = S[:n]
        now *= torch.exp(g[r])[..., None, None]
        new = v[r]
        if beta is not None:
            new = beta[r][..., None] * (new - torch.matmul(k[r][..., None, :], now)[..., 0, :])
        now += k[r][..., None] * new[..., None, :]
        out[r] = s["scale"] * torch.matmul(q[r][..., None, :], now)[..., 0, :]
    return out


def _exact_step(s):
    n = s["batch"] - s["pad"]
    state, at = s["state"].double(), s["index"][:n].long()
    s["first"] = state[at]
    out = _exact_recurrence(s, [torch.arange(n, device=DEV)])
    state[at] = s["first"]
    return {"out": out, "state": state}


def _exact_prompt(s):
    n = _lengths(s["batch"], s["longest"])
    start = [sum(n[:i]) for i in range(len(n))]
    order = sorted(range(len(n)), key=lambda i: -n[i])
    state, at = s["state"].double(), s["index"].long()[torch.tensor(order, device=DEV)]
    s["first"] = state[at] if s["warm"] else torch.zeros_like(state[at])
    begin = torch.tensor([start[i] for i in order], device=DEV)
    left = [n[i] for i in order]
    rows = []
    for t in range(left[0]):
        while left[-1] <= t:
            left.pop()
        rows.append(begin[: len(left)] + t)
    out = _exact_recurrence(s, rows)
    state[at] = s["first"]
    return {"out": out, "state": state}
