"""Cache rows and pages that move, bit for bit against oracle/drafts.py: every other row stays as it was."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import drafts as O
from test_attn_tree_gpu import trees

pytestmark = pytest.mark.gpu


def caches(layers, pages, page, kv, dim, fp8, layout, seed):
    """Host pools per layer [k, v] of raw integers and their PagedKVCaches."""
    rng = np.random.default_rng(seed)
    host, dev = [], []
    dt = torch.uint8 if fp8 else torch.bfloat16
    amax = torch.ones(1, device=DEV) if fp8 else None
    raw = [[rng.integers(0, 256 if fp8 else 1 << 16, (pages, page, kv, dim)).astype(np.uint8 if fp8 else np.uint16)
            for _ in range(2)] for _ in range(layers)]
    up = lambda x: torch.from_numpy(x if fp8 else x.view(np.int16)).to(DEV).view(dt)  # noqa: E731
    if layout == "all layers in a page":                # [pages, layers, 2, page, kv, dim]
        both = torch.stack([torch.stack([up(k), up(v)], 1) for k, v in raw], 1)
        views = [(both[:, i, 0], both[:, i, 1]) for i in range(layers)]
    else:
        views = []
        for k, v in raw:
            k, v = up(k), up(v)
            if layout == "heads first":
                k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
            elif layout == "heads last":                # a gap behind every row, so that nothing is contiguous
                k, v = (torch.nn.functional.pad(x.view(torch.uint8 if fp8 else torch.int16), (0, 32)).view(dt)[..., :dim] for x in (k, v))
            views.append((k, v))
    for (k, v), r in zip(views, raw):
        host.append(r)
        dev.append(nv.PagedKVCache(k, v, amax, amax))
    return host, dev


def same(host, dev, fp8):
    for r, c in zip(host, dev):
        for a, b in zip(r, (c.k, c.v)):
            b = b.cpu().contiguous()
            assert np.array_equal(a, b.numpy() if fp8 else b.view(torch.int16).numpy().view(np.uint16))


LAYOUTS = ["plain", "heads first", "heads last", "all layers in a page"]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,W,kv,dim,page,layers", [(1, 5, 8, 128, 16, 1), (7, 64, 3, 256, 48, 2), (5, 24, 16, 64, 16, 3), (3, 1, 1, 128, 16, 1)])
def test_compact(B, W, kv, dim, page, layers, layout, fp8):
    say(f"[move] compact B={B} W={W} {kv}x{dim} page={page} layers={layers} {layout} fp8={fp8}")
    rng = np.random.default_rng(B * W)
    lens = rng.integers(0, 3 * page, B).astype(np.int32)
    each = -(-(3 * page + W) // page)
    table = rng.permutation(B * each + 2)[: B * each].reshape(B, each).astype(np.int32)
    host, dev = caches(layers, B * each + 2, page, kv, dim, fp8, layout, seed=W)
    parents = trees(B, W, W)
    path, counts = np.full((B, W), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        way = O.way(parents[b], W - 1) if b % 3 else sorted(rng.choice(W, max(1, W // 2), replace=False))
        path[b, : len(way)], counts[b] = way, len(way)
    if B > 4:
        path[3, : W] = rng.permutation(W)                       # any order: all rows change places
        counts[3] = W + 9                                       # clamps
        path[4, 1:3] = [-5, W]                                  # entries that name no node
        table[4, -1] = 1 << 30
        lens[2] = each * page - 2                               # rows behind the table
    O.compact([p for r in host for p in r], table, lens, path, counts)
    to = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    nv.kv_compact(to(table), to(lens), to(path), to(counts), dev if layers > 1 else dev[0])
    torch.cuda.synchronize()
    same(host, dev, fp8)


@pytest.mark.parametrize("lens,counts", [([-3, 5], [4, 4]), ([5, -(1 << 31)], [-1, 4]), ([(1 << 31) - 1, 1 << 30], [4, 4])])
def test_compact_out_of_range(lens, counts):
    host, dev = caches(1, 6, 16, 2, 64, True, "plain", 1)
    table = np.array([[0, 1, 2], [3, -1, 5]], np.int32)
    path = np.array([[3, 2, 1, 0], [0, 2, 3, 1]], np.int32)
    lens, counts = np.array(lens, np.int32), np.array(counts, np.int32)
    O.compact(host[0], table, lens.astype(np.int64), path, counts)
    nv.kv_compact(*(torch.from_numpy(x).to(DEV) for x in (table, lens, path, counts)), dev)
    torch.cuda.synchronize()
    same(host, dev, True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,kv,dim,page,layers", [(1, 8, 128, 64, 1), (5, 3, 256, 48, 2), (2, 1, 64, 16, 4)])
def test_copy_pages(n, kv, dim, page, layers, layout, fp8):
    say(f"[move] copy n={n} {kv}x{dim} page={page} layers={layers} {layout} fp8={fp8}")
    pages = 2 * n + 3
    host, dev = caches(layers, pages, page, kv, dim, fp8, layout, seed=n)
    order = np.random.default_rng(n).permutation(pages).astype(np.int32)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 4:
        src[1], dst[2], src[3], dst[3] = -1, pages, 1 << 30, -(1 << 31)
        src[4] = src[0]                                          # one page to two places
    O.copy_pages([p for r in host for p in r], src, dst)
    nv.kv_copy_pages(torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV), dev)
    torch.cuda.synchronize()
    same(host, dev, fp8)


def test_a_page_onto_itself_and_nothing_to_do():
    host, dev = caches(2, 4, 16, 2, 64, False, "plain", 5)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    nv.kv_copy_pages(i(2, 1), i(2, 1), dev)
    nv.kv_copy_pages(i(), i(), dev)
    nv.kv_compact(torch.zeros(0, 3, dtype=torch.int32, device=DEV), i(), torch.zeros(0, 4, dtype=torch.int32, device=DEV), i(), dev)
    torch.cuda.synchronize()
    same(host, dev, False)


def test_past_two_to_the_31st_element():
    """Rows and pages of a pool of more than 2^31 elements land where they belong."""
    pages, page, kv, dim = 16500, 128, 8, 128
    say(f"[move] a pool of {pages * page * kv * dim} elements")
    amax = torch.ones(1, device=DEV)
    c = nv.PagedKVCache.empty(pages, page, kv, dim, DEV, amax, amax)
    for t, s in ((c.k, 1), (c.v, 2)):
        t.zero_()
        t[-3:].random_(0, 256, generator=torch.Generator(DEV).manual_seed(s))
    last, low = c.k[-1].clone(), c.k[-2].clone()
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    nv.kv_copy_pages(i(pages - 1), i(pages - 3), c)
    assert torch.equal(c.k[-3], last) and torch.equal(c.v[-3], c.v[-1])
    nv.kv_compact(i(pages - 2, pages - 1).view(1, 2), i(126), i(0, 3, -1, -1).view(1, 4), i(2), c)
    torch.cuda.synchronize()
    assert torch.equal(c.k[-2, 127], last[1]) and torch.equal(c.k[-2, :127], low[:127]) and torch.equal(c.k[-1], last)
    assert not c.k[: 100].any() and not c.k[-100:-3].any()


def test_compact_takes_whole_block_tables():
    """A table of which one sequence's row is every sequence's, or whose rows have entries that are not its own
    behind them, is refused: lengths on the device could reach those."""
    host, dev = caches(1, 6, 16, 2, 64, True, "plain", 2)
    wide = torch.arange(12, dtype=torch.int32, device=DEV).reshape(2, 6)
    lens, path, counts = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros((2, 4), dtype=torch.int32, device=DEV), \
        torch.ones(2, dtype=torch.int32, device=DEV)
    for table in (wide[:1].expand(2, 6), wide[:, 2:], wide.t()[:2]):
        with pytest.raises(AssertionError):
            nv.kv_compact(table, lens, path, counts, dev)
    torch.cuda.synchronize()
    same(host, dev, True)
