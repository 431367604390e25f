"""Tree attention over values that are no finite numbers.  Each is one element of one token's value row of one
key-value head: that element of the nodes that attend to the token is then no finite number either, wherever
the token lies (beside drafted tokens, at a window's edge, beside a page outside the pool, in a context's middle).
All other elements and every lse are within the bounds of tests/test_attn_tree_gpu.py."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from oracle import drafts as O
from test_attn_tree_gpu import Case

pytestmark = pytest.mark.gpu


def plant(c, at, seed):
    """Puts a value that is no finite number at rows `at` [(b, row)], each with a key-value head and a column."""
    rng = np.random.default_rng(seed)
    out = []
    for b, row in at:
        page = c.table[b, row // c.page]
        if not 0 <= page < c.cache.num_pages:
            continue
        head, col = int(rng.integers(c.kv)), int(rng.integers(c.dim))
        spot = c.cache.v[int(page), row % c.page, head]
        if c.fp8:
            spot[col] = int(rng.choice([0x7F, 0xFF]))
        else:
            spot[col] = float(rng.choice([np.inf, -np.inf, np.nan]))
        out.append((b, row, head, col))
    return out


def check(c, planted, window=0, scale=None, **kw):
    got = c.run(window=window, scale=scale, **kw)
    torch.cuda.synchronize()
    group = c.heads // c.kv
    reached = np.zeros((len(c.lens), c.W, c.heads, c.dim), bool)
    for b, row, head, col in planted:
        ctx = min(max(int(c.lens[b]), 0), c.max_len)
        for i in range(c.W):
            if row in O.seen(None if c.parents is None else c.parents[b], i, ctx, window):
                reached[b, i, head * group:(head + 1) * group, col] = True
    out = got[0].cpu().double().numpy()
    assert reached.any() and not np.isfinite(out[reached]).any(), f"{np.isfinite(out[reached]).sum()} of {reached.sum()} are finite"
    ref = O.attend(c.qv, *c.pool, c.table, c.lens, c.parents, c.max_len, c.dim ** -0.5 if scale is None else scale, window, c.kv)[0]
    out[reached] = ref[reached]
    c.check((torch.from_numpy(out), got[1]), scale, window)
    return got


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,heads,kv,dim,page", [
    (7, 4, 2, 128, 16), (5, 12, 2, 128, 48), (13, 8, 2, 128, 64), (33, 10, 2, 128, 16), (12, 2, 2, 64, 16), (20, 4, 2, 64, 32),
    (40, 2, 2, 64, 16), (64, 8, 4, 64, 16), (5, 4, 2, 256, 16), (24, 2, 2, 256, 64), (31, 4, 2, 256, 16), (33, 10, 2, 256, 48)])
def test_values_in_any_place(W, heads, kv, dim, page, fp8):
    say(f"[values] W={W} heads={heads}/{kv}x{dim} page={page} fp8={fp8}")
    c = Case([45, 300, 0, 2021, 64, 33], W, heads, kv, dim, page, fp8, seed=W + dim, kind="padded")
    rng = np.random.default_rng(W)
    at = []
    for b, ctx in enumerate(c.lens):
        nodes = [i for i in range(W) if O.way(None if c.parents is None else c.parents[b], i)]
        if nodes:
            at += [(b, int(ctx) + int(i)) for i in rng.choice(nodes, 2)]
            at += [(b, int(r)) for r in (ctx - 1, ctx - 20, rng.integers(0, max(ctx, 1))) if 0 <= r < ctx]
    check(c, plant(c, at, W))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,heads,dim", [(3, 8, 128), (9, 8, 64), (17, 6, 128), (40, 4, 256)])
@pytest.mark.parametrize("window", [3, 50, 333])
def test_values_at_a_windows_edge(window, W, heads, dim, fp8):
    say(f"[values] window={window} W={W} {heads}x{dim} fp8={fp8}")
    c = Case([700, 64, 1501], W, heads, 2, dim, 16, fp8, seed=window, kind="tree")
    at = [(b, int(r)) for b in (0, 1, 2) for r in c.lens[b] + np.array([0, W - 1, -1, 1 - window, W // 2 - window, -window]) if r >= 0]
    check(c, plant(c, at, 3), window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,heads,dim", [(4, 6, 128), (16, 8, 128), (30, 6, 256)])
def test_values_beside_pages_outside_the_pool(W, heads, dim, fp8):
    say(f"[values] pages W={W} {heads}x{dim} fp8={fp8}")
    c = Case([200, 1000], W, heads, 2, dim, 16, fp8, seed=W, kind="chain")
    for b, page, no in ((0, 3, -1), (0, 8, c.cache.num_pages), (1, 40, 1 << 30), (1, 5, -7)):
        c.table[b, page] = no
    c.dev_table = torch.from_numpy(c.table).to(DEV)
    check(c, plant(c, [(0, 33), (0, 40), (0, 70), (0, 150), (1, 64), (1, 659), (1, 90)], 4))


@pytest.mark.parametrize("fp8", [False, True])
def test_values_of_joined_splits(fp8):
    c = Case([9011], 24, 4, 1, 128, 64, fp8, seed=5, kind="tree")
    check(c, plant(c, [(0, 9011), (0, 9010), (0, 4000)], 5))


@pytest.mark.parametrize("fp8", [False, True])
def test_values_that_nobody_sees(fp8):
    """Behind the last node, of a padded node, before a window: nothing is reached."""
    c = Case([90, 41], 10, 8, 2, 128, 16, fp8, seed=6, kind="chain")
    c.parents = np.tile(np.array([-1, 0, 1, -3, 1, 3, 2, 10, 4, 6], np.int32), (2, 1))
    c.dev_parents = torch.from_numpy(c.parents).to(DEV)
    assert len(plant(c, [(0, 100), (0, 93), (1, 41 + 7), (1, 52), (0, 50), (1, 3)], 6)) == 6
    got = c.run(window=20)
    torch.cuda.synchronize()
    c.check(got, window=20)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,heads,dim", [(9, 4, 128), (20, 8, 128), (40, 8, 64), (30, 6, 256)])
def test_values_among_those_of_padded_nodes(W, heads, dim, fp8):
    """Padded nodes' rows that hold no numbers (as they all do here) beside nodes' rows of which one does."""
    say(f"[values] padded W={W} {heads}x{dim} fp8={fp8}")
    c = Case([100, 61, 333], W, heads, 2, dim, 16, fp8, seed=W, kind="chain")
    c.parents = np.tile(np.arange(-1, W - 1, dtype=np.int32), (3, 1))
    c.parents[:, W // 2 + 1:] = -2
    c.dev_parents = torch.from_numpy(c.parents).to(DEV)
    for b in range(3):
        for row in range(int(c.lens[b]) + W // 2 + 1, int(c.lens[b]) + W):
            at = int(c.table[b, row // 16]), row % 16
            for t in (c.cache.k, c.cache.v):
                t[at] = 0x7F if fp8 else float("nan")
    got = c.run()
    torch.cuda.synchronize()
    c.check(got)
    check(c, plant(c, [(0, 100 + W // 2), (2, 333)], W))
