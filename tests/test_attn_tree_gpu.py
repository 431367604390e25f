"""GPU parity of the attention of drafted trees against oracle/drafts.py in 64 bits.

Tolerance, as for the decode attention: scores are off by |ds| <= (D + 4) 2^-24 s, s = scale *
sum |q||k|, and e^x adds 2^-22; a probability is then off by e_p = ds + 2^-22 + w relative, in the
sum over V and in the normaliser, w its rounding: 2^-16 over a bf16 cache (16 significant bits),
2^-11 over E4M3 (fp16), where one below 2^-14 of a row's largest is off by up to 2^-25 of that
instead, n 2^-25 |v| in all.  Sums of n terms add at most (n + 64) 2^-24 of sum p|v|; the result is
rounded to bf16 (2^-8 of itself).  lse is off by ds, w and n 2^-25 (the sum is of the rounded
weights) and one binary32 rounding of itself and of its logarithm."""
import random

import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import drafts as O
from oracle import kvfp8 as F
from oracle import mixers as M

pytestmark = pytest.mark.gpu


def trees(B, W, seed, kind="tree"):
    """Parents [B, W]: random trees, some with padded nodes, forests, or None for chains."""
    if kind == "chain":
        return None
    r = random.Random(seed)
    out = np.zeros((B, W), np.int32)
    for b in range(B):
        for i in range(W):
            out[b, i] = -1 if i == 0 else max(-1, i - 1 - int(r.random() ** 2 * min(i + 1, 9)))
        if kind == "padded" and W > 2:
            for i in r.sample(range(1, W), W // 3):
                out[b, i] = r.choice([-2, i, W + 5, -(1 << 31), (1 << 31) - 1])
    if kind == "padded" and B > 1:
        out[1] = -7
    return out


class Case:
    """A cache, tables and queries on the GPU, and their values on the host.  Rows that no node sees hold NaN."""

    def __init__(self, lens, W, heads, kv, dim, page, fp8, seed=0, layout="plain", max_len=None, kind="tree", gap=0):
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.lens, self.W, self.heads, self.kv, self.dim, self.page, self.fp8 = np.array(lens), W, heads, kv, dim, page, fp8
        self.max_len = max(max(lens), 0) if max_len is None else max_len
        self.parents = trees(B, W, seed, kind)
        need = [-(-(min(max(n, 0), self.max_len) + W) // page) for n in lens]
        pages = sum(need) + 3
        order = rng.permutation(pages)
        self.table = np.full((B, -(-(self.max_len + W) // page) + 1), 1 << 30, np.int32)  # unused entries name no page
        used = np.zeros((pages, page), bool)
        at = 0
        for b, e in enumerate(need):
            self.table[b, :e] = order[at:at + e]
            at += e
            ctx = min(max(lens[b], 0), self.max_len)
            nodes = [i for i in range(W) if O.way(None if self.parents is None else self.parents[b], i)]
            for j in (list(range(ctx)) if nodes else []) + [ctx + i for i in nodes]:
                used[self.table[b, j // page], j % page] = True
        shape = (pages, page, kv, dim)
        if fp8:
            self.amax = [np.float32(4.0), np.float32(3.0)]
            codes = [F.encode(rng.standard_normal(shape).astype(np.float32), a) for a in self.amax]
            for c in codes:
                c[~used] = 0x7F
            self.pool = [F.decode_f32(np.where(used[..., None, None], c, 0), 448.0).astype(np.float64) * (float(a) / 448)
                         for c, a in zip(codes, self.amax)]
            dev = [torch.from_numpy(c).to(DEV) for c in codes]
        else:
            self.amax = [None, None]
            bits = [M.bf16_bits(rng.standard_normal(shape).astype(np.float32)) for _ in range(2)]
            self.pool = [np.where(used[..., None, None], M.bf16_value(b), 0).astype(np.float64) for b in bits]
            for i, b in enumerate(bits):
                b[~used] = (0x7FC0, 0xFF80)[i]
            dev = [torch.from_numpy(b.view(np.int16)).to(DEV).view(torch.bfloat16) for b in bits]
        if layout == "side by side":
            both = torch.stack(dev, 1)
            dev = [both[:, 0], both[:, 1]]
        elif layout == "heads first":
            dev = [d.transpose(1, 2).contiguous().transpose(1, 2) for d in dev]
        self.cache = nv.PagedKVCache(*dev, *[None if a is None else torch.tensor([a], device=DEV) for a in self.amax])
        qb = M.bf16_bits((2 * rng.standard_normal((B, W, heads, dim))).astype(np.float32))
        self.qv = M.bf16_value(qb).astype(np.float64)
        wide = torch.zeros(B, W, heads * dim + gap, dtype=torch.bfloat16, device=DEV)       # rows with a gap between
        wide[..., : heads * dim] = torch.from_numpy(qb.view(np.int16)).to(DEV).view(torch.bfloat16).flatten(2)
        self.q = wide[..., : heads * dim].unflatten(2, (heads, dim))
        self.dev_table = torch.from_numpy(self.table).to(DEV)
        self.dev_lens = torch.from_numpy(self.lens.astype(np.int32)).to(DEV)
        self.dev_parents = None if self.parents is None else torch.from_numpy(self.parents).to(DEV)

    def run(self, **kw):
        kw.setdefault("max_len", self.max_len)
        return nv.attn_tree(self.q, self.cache, self.dev_table, self.dev_lens, self.dev_parents, **kw)

    def check(self, got, scale=None, window=0, what="", skip=None):
        out, lse = (x.cpu().double().numpy() for x in got)
        scale = self.dim ** -0.5 if scale is None else scale
        ref, rl, mag, top = O.attend(self.qv, *self.pool, self.table, self.lens, self.parents, self.max_len, scale, window, self.kv)
        if skip is not None:
            keep = ~skip
            out, lse, ref, rl, mag, top = (x[keep] for x in (out, lse, ref, rl, mag, top))
        ds = (self.dim + 4) * 2.0 ** -24 * top
        n = max(1, max(self.lens) + self.W)
        w, small = (2.0 ** -11, n * 2.0 ** -25) if self.fp8 else (2.0 ** -16, 0.0)
        e = ds + 2.0 ** -22 + w
        tol = 2.0 ** -8 * np.abs(ref) + (2 * e[..., None] + (n + 64) * 2.0 ** -24 + small) * mag + small * 3 + 1e-30
        bad = ~(np.abs(out - ref) <= tol)
        assert not bad.any(), f"{what}: {bad.sum()} outputs off, worst {np.max(np.abs(out - ref) / tol):.2f} of the tolerance"
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), none), f"{what}: empty rows"
        d = np.abs(lse - np.where(none, 0, rl))[~none]
        tl = (ds + (n + 64) * 2.0 ** -24 + w + small + 2.0 ** -22 + 2.0 ** -22 * np.abs(np.where(none, 0, rl)))[~none]
        assert (d <= tl).all(), f"{what}: lse off by {d.max():.2e}"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,heads,kv,dim,page", [
    (1, 40, 8, 128, 64), (5, 24, 4, 256, 16), (16, 16, 16, 64, 48), (3, 48, 2, 128, 16), (33, 3, 1, 64, 32), (2, 1, 1, 256, 128),
    (64, 5, 1, 128, 16), (31, 6, 1, 256, 48), (7, 4, 2, 128, 48), (17, 7, 1, 64, 16), (64, 2, 2, 64, 1024)])
def test_layouts_and_lengths(W, heads, kv, dim, page, fp8):
    lens = [1, 0, 15, 16, 17, 31, 33, 64, 100, 257, 3]
    say(f"[tree] W={W} heads={heads}/{kv}x{dim} page={page} fp8={fp8}")
    c = Case(lens, W, heads, kv, dim, page, fp8, seed=heads + dim + W, kind="padded")
    got = c.run()
    torch.cuda.synchronize()
    c.check(got)


@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("window", [1, 2, 5, 16, 40, 100, 1 << 20])
def test_window(window, kind):
    say(f"[tree] window={window} {kind}")
    c = Case([300, 7, 0, 100, 101, 64], 13, 10, 2, 128, 16, window % 2 == 0, seed=window, kind=kind)
    got = c.run(window=window, scale=0.2)
    torch.cuda.synchronize()
    c.check(got, 0.2, window, f"window {window}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,W,heads,kv,dim,page,window", [
    ([5000], 8, 10, 2, 128, 64, 0), ([4191, 3, 2049, 4096], 5, 5, 1, 128, 16, 0), ([3001, 6000], 20, 4, 2, 256, 128, 0),
    ([9011], 64, 4, 1, 64, 32, 0), ([3000, 5003], 24, 16, 1, 128, 48, 2600), ([2100, 0, 900], 64, 3, 1, 256, 16, 0)])
def test_long_sequences_are_joined(lens, W, heads, kv, dim, page, window, fp8):
    say(f"[tree] long lens={lens} W={W} fp8={fp8}")
    c = Case(lens, W, heads, kv, dim, page, fp8, seed=sum(lens) + W, kind="padded" if len(lens) > 2 else "tree")
    got = c.run(window=window)
    torch.cuda.synchronize()
    c.check(got, window=window)
    again = c.run(window=window)
    torch.cuda.synchronize()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("bound", [2100, 70000])
def test_a_loose_bound_changes_little(bound):
    """The bound of the lengths only chooses the splits."""
    say(f"[tree] loose bound {bound}")
    c = Case([2000, 40, 700], 6, 8, 2, 128, 16, True, seed=3, max_len=2000)
    c.dev_table = torch.nn.functional.pad(c.dev_table, (0, bound // 16 + 1 - c.dev_table.shape[1] + 8), value=-1)
    got = c.run(max_len=bound)
    torch.cuda.synchronize()
    c.check(got)


@pytest.mark.parametrize("layout", ["side by side", "heads first"])
@pytest.mark.parametrize("fp8", [False, True])
def test_cache_layouts_and_strided_queries(layout, fp8):
    say(f"[tree] {layout} fp8={fp8}")
    c = Case([70, 33], 9, 8, 2, 128, 16, fp8, seed=5, layout=layout, gap=64)
    got = c.run()
    torch.cuda.synchronize()
    c.check(got)


def test_lengths_and_pages_out_of_range():
    """Lengths clamp to the bound, pages outside the pool are left out -- the nodes' own among them."""
    say("[tree] out of range")
    c = Case([50, -3, 400, 64], 6, 4, 2, 64, 16, False, seed=8, max_len=90)
    c.table[0, 1] = -1
    c.table[0, 3] = c.cache.num_pages            # the page of nodes 0 .. 5 (rows 50 .. 55)
    c.table[3, 4] = 1 << 30                      # rows 64 .. 69: all the nodes of the last sequence
    c.dev_table = torch.from_numpy(c.table).to(DEV)
    got = c.run()
    torch.cuda.synchronize()
    c.check(got)
    alone = Case([0, 0], 4, 4, 2, 64, 16, False, seed=9)
    alone.table[:] = -1
    alone.dev_table = torch.from_numpy(alone.table).to(DEV)
    out, lse = alone.run()
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_nodes_nan_stays_with_those_that_see_it(fp8):
    """Keys and values of one node that are no numbers: every row that does not see it is unaffected."""
    say(f"[tree] NaN in a node fp8={fp8}")
    c = Case([45, 100], 12, 8, 2, 128, 16, fp8, seed=11)
    skip = np.zeros((2, 12), bool)
    for b, node in ((0, 4), (1, 1)):
        r = c.lens[b] + node
        at = c.table[b, r // 16], r % 16
        for t, x in ((c.cache.k, float("nan")), (c.cache.v, float("inf"))):
            t[int(at[0]), int(at[1])] = 0x7F if fp8 else x
        for i in range(12):
            skip[b, i] = node in O.way(c.parents[b], i)
    assert skip.any() and not skip.all()
    got = c.run()
    torch.cuda.synchronize()
    c.check(got, skip=skip)


def test_a_chain_of_one_equals_the_decode_attention():
    """One node a sequence is the decode attention of one token: the same values within their tolerances."""
    say("[tree] one node")
    c = Case([200, 5000, 1], 1, 16, 2, 128, 16, True, seed=13, kind="chain")
    out, lse = c.run()
    ref, rl = nv.attn_decode(c.q[:, 0], c.cache, c.dev_table, c.dev_lens + 1, max_len=c.max_len + 1)
    torch.cuda.synchronize()
    # each is within 2^-8 of itself of the 64-bit value, and of sum p|v| (|v| <= 3) within some 2^-15 and, the
    # tree's weights being fp16, 2 * 2^-11; its lse is that of the rounded weights
    assert (out[:, 0].double() - ref.double()).abs().le(2 ** -7 * ref.double().abs() + 3 * (2.0 ** -10 + 2.0 ** -13)).all()
    assert torch.allclose(lse[:, 0], rl, rtol=0, atol=2.0 ** -11 + 1e-4)


def test_empty_calls_and_outputs_given():
    c = Case([20, 30], 4, 4, 2, 64, 16, False, seed=14)
    out, lse = nv.attn_tree(c.q[:0], c.cache, c.dev_table[:0], c.dev_lens[:0], c.dev_parents[:0])
    assert out.shape == (0, 4, 4, 64) and lse.shape == (0, 4, 4)
    out, lse = torch.full((2, 4, 4, 64), 7.0, device=DEV).bfloat16(), torch.full((2, 4, 4), 7.0, device=DEV)
    got = c.run(out=out, lse=lse, workspace=nv.Workspace(DEV))
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is lse
    c.check(got)


def test_past_two_to_the_31st_element():
    """Pages of a pool of more than 2^31 elements: the same as from a small pool that holds the same rows."""
    pages, page, kv, D = 16500, 128, 8, 128
    say(f"[tree] a pool of {pages * page * kv * D} elements")
    g = torch.Generator(DEV).manual_seed(6)
    amax = [torch.tensor([4.0], device=DEV) for _ in range(2)]
    big, small = nv.PagedKVCache.empty(pages, page, kv, D, DEV, *amax), nv.PagedKVCache.empty(40, page, kv, D, DEV, *amax)
    far = pages - 1 - 2 * torch.randperm(40, device=DEV, generator=g)
    for a, b in ((big.k, small.k), (big.v, small.v)):
        b.random_(0, 0x70, generator=g)
        a[far] = b
    table = torch.arange(40, device=DEV).view(2, 20)
    lens = torch.tensor([20 * page - 30, 300], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 9, 16, D, device=DEV, generator=g).bfloat16()
    x = nv.attn_tree(q, big, far[table].int(), lens)
    y = nv.attn_tree(q, small, table.int(), lens)
    torch.cuda.synchronize()
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]) and torch.isfinite(x[1]).all()
