"""GPU parity of the decode attention over the paged cache against oracle/mixers.py in 64 bits.

Tolerance.  Scores: products of bf16 (or E4M3) values are exact in binary32 and a sum of D of
them, the scale, the running maximum and the exponential's argument each round by at most 2^-24
of scale * sum |q||k| =: s: |ds| <= (D + 4) 2^-24 s, and e^x adds 2^-22.  Each probability is
thus off by e_p = (D + 4) 2^-24 s + 2^-22 + 2^-16 (its 16 significant bits) relative, both in
the sum over V and in the normaliser; sums of n terms add at most (n + 64) 2^-24 of sum p|v|; the
result is rounded to bf16 (2^-8 of itself).  lse is off by |ds| + e_l, one binary32 rounding of
itself and of its logarithm."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import kvfp8 as F
from oracle import mixers as M

pytestmark = pytest.mark.gpu


class Case:
    """A cache, tables and queries on the GPU, and their values on the host."""

    def __init__(self, lens, heads, kv, dim, page, fp8, seed=0, layout="plain", max_len=None, spare="nan", qscale=2.0):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.kv, self.dim, self.page, self.fp8 = np.array(lens), heads, kv, dim, page, fp8
        B = len(lens)
        self.max_len = max(1, max(lens)) if max_len is None else max_len
        each = -(-max(self.max_len, 1) // page)
        need = [-(-max(min(n, self.max_len), 0) // page) for n in lens]
        pages = sum(need) + 3
        order = rng.permutation(pages)
        self.table = np.full((B, each + 1), 1 << 30, np.int32)     # unused entries name no page
        used = np.zeros((pages, page), bool)
        at = 0
        for b, e in enumerate(need):
            self.table[b, :e] = order[at:at + e]
            for j in range(min(max(lens[b], 0), self.max_len)):
                used[self.table[b, j // page], j % page] = True
            at += e
        shape = (pages, page, kv, dim)
        if fp8:
            self.amax = [np.float32(4.0), np.float32(3.0)]
            codes = [F.encode(rng.standard_normal(shape).astype(np.float32), a) for a in self.amax]
            for c in codes:
                c[~used] = 0x7F                                    # NaN codes in rows nobody attends to
            self.pool = [F.decode_f32(np.where(used[..., None, None], c, 0), 448.0).astype(np.float64) * (float(a) / 448)
                         for c, a in zip(codes, self.amax)]
            dev = [torch.from_numpy(c).to(DEV) for c in codes]
        else:
            self.amax = [None, None]
            bits = [M.bf16_bits(rng.standard_normal(shape).astype(np.float32)) for _ in range(2)]
            self.pool = [np.where(used[..., None, None], M.bf16_value(b), 0).astype(np.float64) for b in bits]
            for i, b in enumerate(bits):
                b[~used] = (0x7FC0, 0x7F80)[i] if spare == "nan" else 0x7F7F
            dev = [torch.from_numpy(b.view(np.int16)).to(DEV).view(torch.bfloat16) for b in bits]
        if layout == "side by side":
            both = torch.stack(dev, 1)
            dev = [both[:, 0], both[:, 1]]
        elif layout == "heads first":
            dev = [d.transpose(1, 2).contiguous().transpose(1, 2) for d in dev]
        self.cache = nv.PagedKVCache(*dev, *[None if a is None else torch.tensor([a], device=DEV) for a in self.amax])
        qb = M.bf16_bits((qscale * rng.standard_normal((B, heads, dim))).astype(np.float32))
        self.qv = M.bf16_value(qb).astype(np.float64)
        self.q = torch.from_numpy(qb.view(np.int16)).to(DEV).view(torch.bfloat16)
        self.dev_table = torch.from_numpy(self.table).to(DEV)
        self.dev_lens = torch.from_numpy(self.lens.astype(np.int32)).to(DEV)

    def run(self, **kw):
        kw.setdefault("max_len", self.max_len)
        return nv.attn_decode(self.q, self.cache, self.dev_table, self.dev_lens, **kw)

    def check(self, got, scale, window=0, what=""):
        out, lse = (x.cpu().double().numpy() for x in got)
        ref, rl, mag, top = M.attend(self.qv, *self.pool, self.table, self.lens, self.max_len, scale, window, self.kv)
        ds = (self.dim + 4) * 2.0 ** -24 * top
        n = max(1, max(self.lens))
        e = ds + 2.0 ** -22 + 2.0 ** -16
        tol = 2.0 ** -8 * np.abs(ref) + (2 * e[..., None] + (n + 64) * 2.0 ** -24) * mag + 1e-30
        bad = np.abs(out - ref) > tol
        assert not bad.any(), f"{what}: {bad.sum()} outputs off, worst {np.max(np.abs(out - ref) / tol):.2f} of the tolerance"
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), none), f"{what}: empty rows"
        d = np.abs(lse - np.where(none, 0, rl))[~none]
        tl = (ds + (n + 64) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -22 * np.abs(np.where(none, 0, rl)))[~none]
        assert (d <= tl).all(), f"{what}: lse off by {d.max():.2e}, tolerance {tl.min():.2e}"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv,dim,page", [(40, 8, 128, 64), (24, 4, 256, 16), (16, 16, 64, 48), (48, 2, 128, 16),
                                               (33, 1, 64, 32), (1, 1, 256, 128), (17, 1, 256, 16)])
def test_layouts_and_lengths(heads, kv, dim, page, fp8):
    lens = [1, 0, 15, 16, 17, 31, 33, 64, 100, 257, 3]
    say(f"[attn] heads={heads}/{kv}x{dim} page={page} fp8={fp8}")
    c = Case(lens, heads, kv, dim, page, fp8, seed=heads + dim)
    got = c.run()
    torch.cuda.synchronize()
    c.check(got, dim ** -0.5)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 1 << 20])
def test_window(window):
    c = Case([300, 7, 0, 100, 101, 64], 10, 2, 128, 16, window % 2 == 0, seed=window)
    got = c.run(window=window, scale=0.2)
    torch.cuda.synchronize()
    c.check(got, 0.2, window, f"window {window}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,heads,kv,dim,page", [
    ([5000], 10, 2, 128, 64), ([8191, 3, 2049, 4096], 5, 1, 128, 16), ([3001, 9000], 4, 2, 256, 128),
    ([20011], 8, 1, 64, 32)])
def test_long_sequences_are_joined(lens, heads, kv, dim, page, fp8):
    say(f"[attn] long lens={lens} fp8={fp8}")
    c = Case(lens, heads, kv, dim, page, fp8, seed=sum(lens))
    got = c.run()
    torch.cuda.synchronize()
    c.check(got, dim ** -0.5)
    again = c.run()
    torch.cuda.synchronize()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1]), "the result depends on timing"


@pytest.mark.parametrize("lens,heads,kv,dim", [
    ([2048, 5, 1024, 700, 1, 2047, 300, 0, 1500], 4, 1, 64),                                  # eight splits
    ([1024, 3, 513, 512, 511, 0, 900, 64, 1, 1000, 700, 17, 256, 1023, 640, 800], 16, 16, 64),  # two
    ([1600, 40, 1599, 0, 900, 533, 534, 1067, 1, 16], 32, 16, 128),                           # four, rows in short supply
    ([1300, 1, 900, 433, 434, 867, 0, 1299], 8, 2, 256)])
def test_uneven_lengths_in_few_splits(lens, heads, kv, dim):
    say(f"[attn] uneven lens={lens}")
    for fp8 in (False, True):
        c = Case(lens, heads, kv, dim, 16, fp8, seed=len(lens))
        got = c.run()
        torch.cuda.synchronize()
        c.check(got, dim ** -0.5)


def test_long_window_and_loose_bound():
    """A bound far above the lengths, and a window whose start lies inside a page and a split."""
    c = Case([6000, 12, 2500, 0], 10, 2, 128, 64, True, seed=3, max_len=40000)
    for window in (0, 3333):
        got = c.run(window=window)
        torch.cuda.synchronize()
        c.check(got, 128 ** -0.5, window, f"window {window}")


def test_lengths_beyond_the_bound_and_negative_ones():
    c = Case([500, -7, 64, 2], 8, 2, 128, 16, False, seed=4, max_len=64)
    got = c.run()
    torch.cuda.synchronize()
    c.check(got, 128 ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_outside_the_pool_are_left_out(fp8):
    c = Case([200, 90, 40], 8, 2, 128, 16, fp8, seed=5)
    c.table[0, 2], c.table[0, 11], c.table[1, 0], c.table[2, :3] = -1, c.cache.num_pages, 1 << 30, -(1 << 31)
    c.dev_table = torch.from_numpy(c.table).to(DEV)
    got = c.run()
    torch.cuda.synchronize()
    c.check(got, 128 ** -0.5)
    assert (got[0][2] == 0).all()


@pytest.mark.parametrize("layout", ["side by side", "heads first"])
@pytest.mark.parametrize("fp8", [False, True])
def test_cache_layouts(layout, fp8):
    c = Case([130, 47, 1], 10, 2, 128, 16, fp8, seed=6, layout=layout)
    got = c.run()
    torch.cuda.synchronize()
    c.check(got, 128 ** -0.5)


def test_large_scores_do_not_overflow():
    """Scores around +-3e4: only differences from the running maximum are exponentiated."""
    c = Case([700, 65], 8, 2, 128, 16, False, seed=7, qscale=200.0)
    for scale in (13.0, -13.0, 0.0):
        got = c.run(scale=scale)
        torch.cuda.synchronize()
        c.check(got, scale, what=f"scale {scale}")


def test_infinite_keys_take_no_weight_or_all():
    """A key of -inf against a positive query has probability 0; the rest is as without it."""
    c = Case([40], 2, 1, 64, 16, False, seed=8)
    c.q.abs_()
    c.qv = np.abs(c.qv)
    ref = Case([40], 2, 1, 64, 16, False, seed=8)
    ref.q.abs_()
    c.cache.k[c.table[0, 1], 3] = -float("inf")
    ref.cache.v[c.table[0, 1], 3] = 0
    got = c.run(window=0)
    torch.cuda.synchronize()
    kp = c.pool[0].copy()
    kp[c.table[0, 1], 3] = -1e30
    o, l, _, _ = M.attend(c.qv, kp, c.pool[1], c.table, c.lens, c.max_len, 0.125, 0, 1)
    assert np.allclose(got[0].cpu().double().numpy(), o, rtol=2.0 ** -7, atol=1e-3)
    assert np.allclose(got[1].cpu().double().numpy(), l, atol=1e-4)


def test_strided_queries_outputs_and_rows_left_alone():
    c = Case([70, 33], 10, 2, 128, 16, True, seed=9)
    wide = torch.full((2, 12, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    qw = torch.zeros((2, 20, 128), dtype=torch.bfloat16, device=DEV)
    qw[:, 5:15] = c.q
    lse = torch.empty((2, 10), device=DEV)
    out, _ = nv.attn_decode(qw[:, 5:15], c.cache, c.dev_table, c.dev_lens, max_len=c.max_len, out=wide[:, 1:11], lse=lse)
    torch.cuda.synchronize()
    c.check((out, lse), 128 ** -0.5)
    assert (wide[:, 0] == 7).all() and (wide[:, 11] == 7).all()


def test_refusals():
    c = Case([70, 33], 10, 2, 128, 16, True, seed=9)
    with pytest.raises(AssertionError):
        c.run(max_len=10000)
    with pytest.raises(AssertionError):
        nv.attn_decode(c.q.float(), c.cache, c.dev_table, c.dev_lens)
    with pytest.raises(AssertionError):
        nv.attn_decode(c.q, c.cache, c.dev_table.long(), c.dev_lens)
    with pytest.raises(AssertionError):
        nv.attn_decode(c.q, c.cache, c.dev_table, c.dev_lens[:1])
    with pytest.raises(nv.NVFP4Error):
        nv.attn_decode(c.q[:, :9], c.cache, c.dev_table, c.dev_lens)
    with pytest.raises(nv.NVFP4Error):                     # one row of pages for all: its stride is 0
        nv.attn_decode(c.q, c.cache, c.dev_table[:1].expand(2, -1), c.dev_lens)
    with pytest.raises(nv.NVFP4Error):
        c.run(scale=float("nan"))
    with pytest.raises(TypeError):
        c.run(stream=5)
