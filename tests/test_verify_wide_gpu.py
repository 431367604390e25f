"""Verification over vocabularies of more than 16 chunks of 8192 logits, which several threads of a node take in
turns, and of more than 64, of which a lane takes several in the draw.  Against oracle/drafts.py in 64 bits;
tokens, paths and counts are equal where no decision lies within 2^-36 of a border (of the last draw after a
rejection: in the unnormalised weights max(p - q, 0), whose total may be small)."""
import numpy as np
import pytest

from gpu_util import say
from test_verify_gpu import _case, _check, _run

pytestmark = pytest.mark.gpu

FAR = 16 * 8192         # the first logit of the second turn
WIDE = [131073, 151936, 262147, 600001]


def _far_ends(c, seed):
    """Peaks, drafts and most of the weight in the last chunks for half of the sequences, in the first for the others."""
    rng = np.random.default_rng(seed)
    B, W, V = c["logits"].shape
    inner = np.arange(-1, W - 1)
    for b in range(B):
        lo, hi = (FAR, V) if b % 2 else (0, V)
        for x in (c["logits"], c["draft_logits"]):
            if x is not None:
                x[b, :, lo:hi] += np.float32(3)
                x[b, :, rng.integers(lo, hi)] = np.float32(np.log(V) + 5)
        if c["draft_logits"] is not None:
            heat = c["temperature"][b] if c["temperature"][b] > 0 else 1
            for i in range(1, W):
                c["drafts"][b, i] = (c["draft_logits"][b, inner[i]] / heat + rng.gumbel(size=V)).argmax()
        else:
            up = inner if c["parents"] is None else c["parents"][b]
            for i in range(1, W):
                c["drafts"][b, i] = rng.integers(lo, hi)
                if 0 <= up[i] < W:
                    c["logits"][b, up[i], c["drafts"][b, i]] = np.float32(np.log(V) + 6 + rng.standard_normal())
    return c


@pytest.mark.parametrize("V", WIDE)
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_picked_drafts(V, kind):
    say(f"[wide] picked V={V} {kind}")
    c = _far_ends(_case(6, 4, V, seed=V, kind=kind, greedy=2), V)
    tokens, _, counts = got = _run(c)
    assert _check(c, got) > 0
    assert (tokens >= FAR).any()


@pytest.mark.parametrize("V", WIDE)
def test_drawn_drafts(V):
    say(f"[wide] drawn V={V}")
    c = _far_ends(_case(6, 4, V, seed=V + 1, kind="chain", sampled=True, greedy=1), V)
    tokens, _, counts = got = _run(c)
    assert _check(c, got) > 0
    assert (tokens >= FAR).any() and (counts < 4).any()


@pytest.mark.parametrize("V", WIDE)
def test_one_sequence_of_many_nodes(V):
    say(f"[wide] nodes V={V}")
    c = _far_ends(_case(1, 33, V, seed=V + 2), V)
    _check(c, _run(c))


@pytest.mark.parametrize("V", [262147, 600001])
def test_largest_logits_that_are_equal(V):
    """Equal largest logits in chunks that one thread takes in turns, and in those of two threads: the lowest index."""
    say(f"[wide] ties V={V}")
    rng = np.random.default_rng(V)
    c = _case(12, 2, V, seed=5, kind="chain", greedy=12)
    want = []
    for b in range(12):
        chunk, step = int(rng.integers(0, 16)), (1, 5, 16)[b % 3]
        at = np.array([chunk, chunk + step]) * 8192 + rng.integers(0, 8192, 2)
        at = np.minimum(at, V - 1)
        c["logits"][b, :, at] = 50.0
        c["drafts"][b, 1] = at.min() if b % 2 else at.max()
        want.append(at.min())
    tokens, _, counts = got = _run(c)
    _check(c, got)
    assert list(tokens[:, 0]) == want and list(counts) == [2 if b % 2 else 1 for b in range(12)]


@pytest.mark.parametrize("V", [262147, 600001])
def test_filtered_rows(V):
    """A few tokens left, far from each other: the children are turned down, the last token is one of the rest."""
    say(f"[wide] filtered V={V}")
    rng = np.random.default_rng(V)
    c = _case(20, 3, V, seed=6, kind="chain")
    c["logits"][:] = -np.inf
    for b in range(20):
        for i in range(3):
            kept = np.unique(rng.integers(0, V, 7))
            c["logits"][b, i, kept] = rng.standard_normal(len(kept))
            if i < 2:
                c["drafts"][b, i + 1] = rng.choice(kept)
    c["uniforms"][:, 0] = np.where(np.arange(20) % 3 == 0, 0.99, c["uniforms"][:, 0])
    c["uniforms"][::2, 3] = 0
    _check(c, _run(c))
