"""Which paged caches the library takes: no row of k may overlap a row of v, wherever in one
allocation they lie, or an append would write one over the other.  A call of no tokens checks the
cache and launches nothing."""
import ctypes

import numpy as np
import pytest

import nvfp4_w4a4_block_act_amd as nv

A = 1 << 40


def status(v_bytes, pages, page, heads, dim, strides, elem=2):
    """The append's status for a cache whose v lies v_bytes behind k; strides of page, token, head in elements."""
    c = nv.KVCacheDesc(A, A + v_bytes, A - 4096 if elem == 1 else None, A - 2048 if elem == 1 else None, pages, *strides, page,
                       heads, dim, 2 if elem == 1 else 1)
    return nv.lib().nvfp4_kv_append(None, None, None, 1, 0, 0, 0, heads * dim, heads * dim, None, 0, 0, 0, None, None,
                                    ctypes.byref(c), None, 0, None)


def meet(v, pages, page, heads, dim, strides):
    """Whether a row of k meets one of v, v elements behind it, from all of their elements."""
    at = (np.arange(pages)[:, None, None] * strides[0] + np.arange(page)[:, None] * strides[1] + np.arange(heads) * strides[2])
    k = (at.reshape(-1, 1) + np.arange(dim)).ravel()
    assert len(np.unique(k)) == k.size
    return bool(np.isin(k + v, k).any())


def test_named_layouts():
    page = 16 * 8 * 128
    whole = (page, 8 * 128, 128)
    for v, strides, want in [
            (2 * 32 * page, whole, 0),                                  # one behind the other
            (2 * 32 * page - 16, whole, 1),                             # the last row's end is the first one's start
            (16, whole, 1), (2 * 128, whole, 1), (2 * page, whole, 1),  # a head, a page further
            (2 * page, (2 * page, 8 * 128, 128), 0),                    # pages side by side
            (2 * 8 * 128, (2 * page, 2 * 8 * 128, 128), 0),             # tokens side by side
            (2 * 128, (2 * page, 2 * 8 * 128, 256), 0),                 # heads side by side
            (2 * 64, (2 * page, 2 * 8 * 128, 256), 1),                  # half a head into them
            (2 * 3 * page, (2 * page, 8 * 128, 128), 0), (2 * 4 * page, (2 * page, 8 * 128, 128), 1),
            (2 * 63 * page, (2 * page, 8 * 128, 128), 0), (2 * 64 * page, (2 * page, 8 * 128, 128), 0)]:
        assert status(v, 32, 16, 8, 128, strides) == want, (v, strides)
        assert status(-v, 32, 16, 8, 128, strides) == want, (-v, strides)
        assert status(v // 2, 32, 16, 8, 128, strides, elem=1) == (want if v % 32 == 0 else 3), (v, strides, "codes")


@pytest.mark.parametrize("seed", range(6))
def test_any_layout_against_all_elements(seed):
    rng = np.random.default_rng(seed)
    seen = set()
    for _ in range(150):
        pages, page, heads, dim = int(rng.integers(1, 4)), 16 * int(rng.integers(1, 3)), int(rng.integers(1, 4)), 64
        counts = {"page": pages, "token": page, "head": heads}
        span, stride = dim, {}
        for name in rng.permutation(list(counts)):                      # any order of the axes, with gaps
            stride[name] = span + 8 * int(rng.integers(0, 30)) * int(rng.integers(0, 2))
            span += (counts[name] - 1) * stride[name] if counts[name] > 1 else 0
        strides = tuple(stride[n] for n in ("page", "token", "head"))
        v = 8 * int(rng.integers(1, span // 8 + 20)) * int(rng.choice([-1, 1]))
        want = meet(v, pages, page, heads, dim, strides)
        seen.add(want)
        assert status(2 * v, pages, page, heads, dim, strides) == int(want), (v, pages, page, heads, strides)
    assert seen == {True, False}


def test_far_apart_and_empty_caches():
    big = (1 << 40) - 8
    assert status((1 << 60) + 16, 1 << 16, 16, 8, 128, (big, 1024, 128)) == 0
    assert status(2 * big * 7 + 256, 1 << 16, 16, 8, 128, (big, 1024, 128)) == 1
    assert status(2 * big * 7 + 2 * 16 * 1024, 1 << 16, 16, 8, 128, (big, 1024, 128)) == 0
    assert status(16, 0, 16, 8, 128, (16 * 1024, 1024, 128)) == 0
