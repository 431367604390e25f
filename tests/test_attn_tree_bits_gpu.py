"""Tree attention over E4M3 keeps as many bits of a probability as over bf16 and as the decode attention:
16, whatever its size.  The bounds are those of tests/test_attn_tree_gpu.py with w = 2^-16 and no term
for small probabilities (its bounds for a bf16 cache)."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import kvfp8 as F
from test_attn_tree_gpu import Case

pytestmark = pytest.mark.gpu


def check(c, **kw):
    got = c.run(**kw)
    torch.cuda.synchronize()
    c.fp8 = False                       # the bounds of 16 bits
    c.check(got, kw.get("scale"), kw.get("window", 0))


@pytest.mark.parametrize("scale", [None, 1.0, -0.7])
@pytest.mark.parametrize("W,heads,kv,dim,page", [
    (1, 40, 8, 128, 64), (5, 24, 4, 256, 16), (16, 16, 16, 64, 48), (3, 48, 2, 128, 16), (33, 3, 1, 64, 32), (2, 1, 1, 256, 128),
    (64, 5, 1, 128, 16), (31, 6, 1, 256, 48), (7, 4, 2, 128, 48), (17, 7, 1, 64, 16), (64, 2, 2, 64, 1024)])
def test_bits_of_the_weights(W, heads, kv, dim, page, scale):
    say(f"[bits] W={W} heads={heads}/{kv}x{dim} scale={scale}")
    check(Case([1, 0, 15, 16, 17, 31, 33, 64, 100, 257, 3], W, heads, kv, dim, page, True, seed=dim + W, kind="padded"), scale=scale)


@pytest.mark.parametrize("lens,W,heads,kv,dim,window", [([5000], 8, 10, 2, 128, 0), ([9011], 64, 4, 1, 64, 0), ([2100, 0, 900], 64, 3, 1, 256, 333)])
def test_bits_over_joined_splits(lens, W, heads, kv, dim, window):
    say(f"[bits] lens={lens}")
    check(Case(lens, W, heads, kv, dim, 32, True, seed=W, kind="tree"), window=window)


def test_one_node_against_the_decode_attention():
    """Each is within 2^-8 of itself and some 2^-15 of sum p|v| (|v| <= 3) of the 64-bit value."""
    c = Case([200, 5000, 1, 7000], 1, 16, 2, 128, 16, True, seed=13, kind="chain")
    out, lse = c.run()
    ref, rl = nv.attn_decode(c.q[:, 0], c.cache, c.dev_table, c.dev_lens + 1, max_len=c.max_len + 1)
    torch.cuda.synchronize()
    assert (out[:, 0].double() - ref.double()).abs().le(2 ** -7 * ref.double().abs() + 6 * 2.0 ** -14).all()
    assert torch.allclose(lse[:, 0], rl, rtol=0, atol=1e-4)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_small_weights(dim):
    """One token with almost all of the weight and a value of 0, and n = 2^17 - 64 others, each with 2^-25.5 of
    its weight, whose values alone make the result, 3 n 2^-25.5 = 0.008.  In one split (enough workgroups to fill the GPU), the large one first.
    Bounds: each small probability to e = (dim + 4) 2^-24 * 18 + 2^-22 + 2^-16, the sums of n terms to n 2^-24,
    the result to 2^-8."""
    W, kv, group, B, page, n = 64, 8, 16, 24, 1024, 2 ** 17 - 64
    say(f"[bits] {n} small weights, heads of {dim}")
    amax = torch.tensor([3.0], device=DEV)
    cache = nv.PagedKVCache.empty(2 ** 17 // page, page, kv, dim, DEV, amax, amax)
    cache.k.zero_()
    cache.v.fill_(int(F.encode(np.full((1, 1), 3.0, np.float32), np.float32(3.0)).flat[0]))
    cache.k[0, 0, :, 0] = int(F.encode(np.full((1, 1), 3.0, np.float32), np.float32(3.0)).flat[0])
    cache.v[0, 0] = 0
    q = torch.zeros(B, W, kv * group, dim, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    scale = 25.5 * float(np.log(2)) / 3.0
    table = torch.arange(2 ** 17 // page, dtype=torch.int32, device=DEV).repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    parents = torch.zeros(B, W, dtype=torch.int32, device=DEV)
    parents[:, 0] = -1                                                   # each node sees the context, node 0 and itself
    assert nv.nvfp4_attn_tree_workspace_bytes(B, W, kv * group, kv, dim, n, 0) == 0, "the sequences have to be one split each"
    out, lse = nv.attn_tree(q, cache, table, lens, parents, max_len=n, scale=scale)
    torch.cuda.synchronize()
    seen = n - 1 + torch.where(torch.arange(W, device=DEV) == 0, 1.0, 2.0).double()
    small = seen * 2.0 ** -25.5
    want = (3 * small / (1 + small))[None, :, None, None]
    e = 2 * ((dim + 4) * 2.0 ** -24 * 18 + 2.0 ** -22 + 2.0 ** -16) + (n + 64) * 2.0 ** -24
    off = ((out.double() - want).abs() / want).max().item()
    assert off <= 2.0 ** -8 + e, f"off by {off:.4f} of the result"
    assert ((lse.double() - (scale * 3 + torch.log1p(small))[None, :, None]).abs() <= (dim + 4) * 2.0 ** -24 * 18 + (n + 64) * 2.0 ** -24).all()
