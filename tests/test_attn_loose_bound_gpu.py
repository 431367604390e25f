"""Decode attention under a bound far above the lengths, as a captured graph or the default bound
(what the block table holds) gives it: a sequence's splits follow its own length, which must come
out right wherever it lies below the bound.  (That a loose bound leaves as many workgroups at work
as a tight one is checked on the CPU, tests/abi_host/check_attn_splits.cpp.)  Tolerances are those
of test_attn_decode_gpu.py."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from test_attn_decode_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,heads,kv,dim", [([5000], 40, 8, 128), ([4500, 20, 0, 4777], 8, 4, 64), ([9000], 6, 2, 256)])
def test_bounds_far_above_the_lengths(lens, heads, kv, dim, fp8):
    say(f"[attn] loose bounds lens={lens} fp8={fp8}")
    for bound in (max(lens), 2 * max(lens) - 1, 2 * max(lens), 1 << 15, 1 << 17, 1 << 20):
        c = Case(lens, heads, kv, dim, 64, fp8, seed=7, max_len=bound)
        got = c.run()
        torch.cuda.synchronize()
        c.check(got, dim ** -0.5, what=f"bound {bound}")
        again = c.run()
        torch.cuda.synchronize()
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1]), "the result depends on timing"


@pytest.mark.parametrize("window", [0, 1, 700, 3000, 1 << 30])
def test_windows_under_a_loose_bound(window):
    c = Case([6000, 12, 2500, 0, 701, 3001], 10, 2, 128, 16, window % 2 == 0, seed=8, max_len=1 << 16)
    got = c.run(window=window)
    torch.cuda.synchronize()
    c.check(got, 128 ** -0.5, window, f"window {window}")


def test_one_long_sequence_in_a_large_batch():
    for B, where in ((65, 64), (130, 127), (200, 0), (200, 199)):
        lens = list(np.random.default_rng(B + where).integers(0, 60, B))
        lens[where] = 3111
        c = Case([int(n) for n in lens], 2, 1, 64, 16, True, seed=B, max_len=8000)
        got = c.run()
        torch.cuda.synchronize()
        c.check(got, 0.125, what=f"{B} sequences, the longest at {where}")


def test_lengths_above_the_bound_in_a_split_batch():
    c = Case([5000, -3, 9000, 4100], 8, 2, 128, 16, False, seed=9, max_len=4100)
    got = c.run()
    torch.cuda.synchronize()
    c.check(got, 128 ** -0.5)


def test_growing_lengths_in_one_graph():
    """One captured call under a loose bound, replayed while the sequences grow over the lengths
    where they get more splits: every replay against the call under a tight bound."""
    c = Case([4200, 3000], 8, 2, 128, 64, True, seed=10, max_len=1 << 15)
    lens = c.dev_lens
    out, lse = c.run()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.run(out=out, lse=lse)
    for n in (1, 500, 1023, 1024, 1025, 1600, 2048, 4200, 0):
        lens[0], lens[1] = n, max(0, n - 1200)
        c.lens[:] = n, max(0, n - 1200)
        out.fill_(float("nan")), lse.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        (torch.ones(4, device=DEV) + 1).sum().item()
        torch.cuda.synchronize()
        c.check((out, lse), 128 ** -0.5, what=f"length {n}")
