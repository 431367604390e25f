"""Tree attention where a wave takes more than 32 turns, for which it looks the pages up anew, with pages outside
the pool, a window's edge and values that are no finite numbers around the 32nd; and joins of more than eight
splits of many rows.  Bounds: those of tests/test_attn_tree_gpu.py for weights of 16 bits.

Splits are long where many workgroups run: the sequences of a case are attended to many times over in one
call, and all of these give the same."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import drafts as O
from test_attn_tree_gpu import Case
from test_attn_tree_values_gpu import check as check_values
from test_attn_tree_values_gpu import plant

pytestmark = pytest.mark.gpu


class Repeated(Case):
    """The sequences of a case `times` times over; the first ones' results."""
    times = 1

    def splits(self, window=0):
        B = len(self.lens) * self.times
        need = nv.nvfp4_attn_tree_workspace_bytes(B, self.W, self.heads, self.kv, self.dim, self.max_len, window)
        return max(1, need // (B * self.W * self.heads * (self.dim + 2) * 4))

    def run(self, **kw):
        kw.setdefault("max_len", self.max_len)
        n, r = len(self.lens), self.times
        out, lse = nv.attn_tree(self.q.repeat(r, 1, 1, 1), self.cache, self.dev_table.repeat(r, 1), self.dev_lens.repeat(r),
                                self.dev_parents.repeat(r, 1), **kw)
        torch.cuda.synchronize()
        bits, sums = out.view(torch.int16).view(r, n, -1), lse.view(torch.int32).view(r, n, -1)
        assert (bits == bits[:1]).all() and (sums == sums[:1]).all()
        return out[:n], lse[:n]


def case(W, heads, kv, dim, fp8, lens, groups, window=0, kind="tree"):
    """A case whose waves take more than 33 turns in tiles of 32 tokens, `groups` of them in turn."""
    c = Repeated(lens, W, heads, kv, dim, 16, fp8, seed=W + dim, kind=kind)
    blocks = -(-W * heads // kv // 128)
    c.times = -(-1536 // (len(lens) * kv * blocks))
    first = [max(0, (n - window) // 32 * 32) if window else 0 for n in lens]
    span = max(n + W - f for n, f in zip(lens, first))
    assert span / c.splits(window) > 33 * 32 * groups
    return c, first


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 1])
@pytest.mark.parametrize("W,heads,dim,groups", [
    (16, 8, 64, 1), (16, 8, 128, 1), (16, 8, 256, 1), (30, 8, 64, 1), (30, 8, 128, 1), (30, 8, 256, 1), (4, 8, 64, 4), (4, 8, 128, 4),
    (4, 8, 256, 4), (8, 8, 64, 4), (8, 8, 128, 4), (8, 8, 256, 2)])
def test_pages_around_the_32nd_turn(W, heads, dim, groups, window, fp8):
    far = 1200 * groups
    lens = [far + 37, far + 900, far - 40]
    window = window * (far - 55)
    say(f"[turns] W={W} {heads}/2x{dim} groups={groups} window={window} fp8={fp8}")
    c, first = case(W, heads, 2, dim, fp8, lens, groups, window)
    for b, f in enumerate(first):
        for k in {1, groups}:                            # (waves that share tiles, and that take them in turn)
            for i, at in enumerate([1024 * k - 40, 1024 * k + 5, 1024 * k + 30 * (b + 1)]):
                c.table[b, (f + at) // 16] = (-1, c.cache.num_pages, 1 << 30)[i]
        if window:                                       # no numbers right before the first token that anybody sees
            row = int(c.lens[b]) - window
            at = int(c.table[b, row // 16]), row % 16
            for t in (c.cache.k, c.cache.v):
                t[at] = 0x7F if fp8 else float("nan")
    c.dev_table = torch.from_numpy(c.table).to(DEV)
    got = c.run(window=window)
    c.fp8 = False                                        # the bounds of 16 bits
    c.check(got, window=window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("W,heads,dim,groups", [(16, 8, 128, 1), (30, 8, 256, 1), (30, 8, 128, 1), (4, 8, 128, 4), (8, 8, 64, 4)])
def test_values_around_the_32nd_turn(W, heads, dim, groups, fp8):
    """Values that are no finite numbers, in tiles that half of a page outside the pool makes masked ones."""
    say(f"[turns] values W={W} {heads}/2x{dim} groups={groups} fp8={fp8}")
    far = 1200 * groups
    c, _ = case(W, heads, 2, dim, fp8, [far + 37, far + 211], groups)
    at = []
    for b in range(2):
        for k in {1, groups}:
            for tile in (31, 32, 33):
                token = tile * 32 * k + 32 * b
                c.table[b, token // 16 + 1] = -1
                at.append((b, token + 7))
    c.dev_table = torch.from_numpy(c.table).to(DEV)
    check_values(c, plant(c, at + [(0, int(c.lens[0]) + 1)], W))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim,lens,kind", [(64, [10000, 9001], "tree"), (128, [7000, 5100], "padded"), (256, [5000, 4700], "tree")])
def test_joins_of_many_rows(dim, lens, kind, fp8):
    say(f"[turns] joins {lens} heads of {dim} fp8={fp8}")
    c = Repeated(lens, 64, 16, 1, dim, 64, fp8, seed=dim, kind="tree")
    if kind == "padded":
        c.parents[0, 5:9] = -2
        c.dev_parents = torch.from_numpy(c.parents).to(DEV)
        assert any(not O.way(c.parents[0], i) for i in range(9, 64))
    assert c.splits() > 8 and len(lens) * 64 * 16 >= 2048
    got = c.run()
    c.fp8 = False
    c.check(got)


@pytest.mark.parametrize("W,heads,kv,dim,lens", [(64, 16, 2, 256, [9000]), (30, 32, 4, 128, [4300]), (12, 16, 2, 64, [20000]), (50, 8, 1, 256, [6000, 2500])])
def test_joins_of_fewer_rows(W, heads, kv, dim, lens):
    """Joins by four and by sixteen sets of lanes a row: up to 2047 rows of more than eight splits."""
    c = Repeated(lens, W, heads, kv, dim, 64, False, seed=W, kind="tree")
    say(f"[turns] joins {lens} {W * heads * len(lens)} rows of {dim} in {c.splits()} splits")
    assert c.splits() > 8 and len(lens) * W * heads < 2048
    c.check(c.run())
