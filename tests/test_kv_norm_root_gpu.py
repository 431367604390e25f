"""The norm's factor, bit for bit.  Elements are small whole numbers, so that a head's sum of squares and its
mean are exact in binary32 in every order of the additions: 1 / sqrt(mean + eps) has one value of two
roundings, and y = (x * factor) * w, rounded to bf16, one more each."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import mixers as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -10])
def test_the_factor_is_rounded_like_a_root_and_a_division(dim, eps):
    say(f"[root] heads of {dim}, eps {eps}")
    rng = np.random.default_rng(dim)
    T, heads, page = 4000, 8, 16
    x = rng.integers(1, 9, (T, heads, dim)) * rng.choice([-1, 1], (T, heads, dim))
    w = (1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)
    dx = torch.from_numpy(x.astype(np.float32)).to(DEV)
    cache = nv.PagedKVCache.empty(T // page, page, 1, dim, DEV)
    slots = torch.arange(T, device=DEV)
    q = nv.kv_append(dx[:, :1].contiguous(), dx[:, :1].contiguous(), cache, slots, q=dx, q_norm=torch.from_numpy(w).to(DEV),
                     k_norm=torch.from_numpy(w).to(DEV), eps=eps)
    torch.cuda.synchronize()
    mean = ((x.astype(np.int64) ** 2).sum(-1, keepdims=True) / dim + eps).astype(np.float32)
    factor = np.float32(1) / np.sqrt(mean)
    assert factor.dtype == np.float32
    bits = M.bf16_bits((x.astype(np.float32) * factor) * w)
    got = q.cpu().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(got, bits), f"{(got != bits).sum()} of {bits.size} queries differ"
    keys = cache.k.view(T, dim).cpu().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(keys, bits[:, 0])
