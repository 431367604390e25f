"""Heads whose squares lie below binary32's range, with no eps or one as small: normed like any other.
Against oracle/drafts.py in 64 bits, the tolerance as in tests/test_kv_norm_gpu.py: 20 * 2^-24 of the value for
the sum, the root and the products, then 2^-8 for bf16."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import drafts as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 3e-38, 1e-33, 7e-31, 1e-20, 1e-6])
def test_small_heads(eps, src, dim):
    say(f"[small] heads of {dim}, {src}, eps {eps}")
    rng = np.random.default_rng(dim)
    sizes = np.array([1e-10, 3e-15, 1e-16, 1e-18, 1e-19, 1e-20, 1e-22, 1e-25, 1e-30, 1e-36, 1e-38, 1e-40, 1e-43, 0.0])
    T, heads, page = 16 * len(sizes), 3, 16
    x = rng.standard_normal((T, heads, dim)) * np.repeat(sizes, 16)[:, None, None]
    x[::3, 1] *= 1e7                                        # heads of one wave that differ
    x[1::5, 2, rng.integers(0, dim)] *= 1e6                 # one large element in a small head
    dt = torch.float32 if src == "f32" else torch.bfloat16
    host = torch.from_numpy(x.astype(np.float32)).to(dt)
    x = host.double().numpy()
    w = (1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)
    dx, dw = host.to(DEV), torch.from_numpy(w).to(DEV)
    cache = nv.PagedKVCache.empty(T // page, page, 1, dim, DEV)
    q = nv.kv_append(dx[:, :1].contiguous(), dx[:, 1:2].contiguous(), cache, torch.arange(T, device=DEV), q=dx, q_norm=dw, k_norm=dw, eps=eps)
    torch.cuda.synchronize()
    y = O.norm(x, w.astype(np.float64), float(np.float32(eps)))
    tol = (2.0 ** -8 + 20 * 2.0 ** -24) * np.abs(y) + 1e-38
    off = np.abs(q.double().cpu().numpy() - y)
    assert (off <= tol).all(), f"{(off > tol).sum()} of {y.size} off, worst {(off / tol).max():.1f} of the tolerance"
    keys = cache.k.view(T, dim).double().cpu().numpy()
    assert (np.abs(keys - y[:, 0]) <= tol[:, 0]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_an_element_that_is_no_finite_number(bad):
    """By the formula a head that holds NaN is NaN throughout; one that holds an infinity is NaN there and 0
    elsewhere.  Other heads are what they were."""
    g = torch.Generator(DEV).manual_seed(1)
    x, w = torch.randn(32, 5, 128, device=DEV, generator=g), torch.rand(128, device=DEV, generator=g) + 0.5
    spoilt = x.clone()
    spoilt[3, 2, 40] = spoilt[17, 0, 127] = spoilt[31, 4, 0] = bad
    got = []
    for a in (x, spoilt):
        cache = nv.PagedKVCache.empty(2, 16, 5, 128, DEV)
        q = nv.kv_append(a, a, cache, torch.arange(32, device=DEV), q=a, q_norm=w, k_norm=w)
        got.append((q.float().cpu(), cache.k.view(32, 5, 128).float().cpu()))
    torch.cuda.synchronize()
    heads, at = ([3, 17, 31], [2, 0, 4]), ([3, 17, 31], [2, 0, 4], [40, 127, 0])
    for good, out in zip(*got):
        kept = torch.ones(32, 5, dtype=torch.bool)
        kept[heads] = False
        assert torch.equal(out[kept], good[kept])
        assert torch.isnan(out[at]).all()
        rest = torch.ones(32, 5, 128, dtype=torch.bool)
        rest[at] = False
        inside = out[rest & ~kept[..., None]]
        assert torch.isnan(inside).all() if bad != bad else (inside == 0).all()
