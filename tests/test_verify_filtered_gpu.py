"""Verification over filtered logits (-inf for all but a few tokens): a token without a weight is never
drawn, whatever the last uniform number.  Against oracle/drafts.py in 64 bits; tokens, paths and counts are
equal where no decision lies within 2^-36 of a border."""
import numpy as np
import pytest

from gpu_util import say
from test_verify_gpu import _check, _run

pytestmark = pytest.mark.gpu

CHUNK = 8192            # logits that the kernels sum at a time


def _chain(V, B, W=2):
    return dict(logits=np.full((B, W, V), -np.inf, np.float32), drafts=np.zeros((B, W), np.int64), parents=None,
                temperature=np.ones(B, np.float32), uniforms=np.full((B, W + 1), 0.5, np.float32), draft_logits=None)


def _as_counted(c):
    """The same numbers as the definition counts them: below 0 and NaN as 0."""
    return dict(c, uniforms=np.clip(np.nan_to_num(c["uniforms"], nan=0), 0, None).astype(np.float32))


@pytest.mark.parametrize("V,child,other", [(16384, 7, 9000), (20000, 10, 9000), (8192 + 9, 8191, 8192), (3 * CHUNK, 9000, 5),
                                           (100003, 4, 99999), (9000, 40, 41)])
def test_a_rejected_token_alone_in_its_chunk(V, child, other):
    """Two tokens are left; the child is turned down, so that the last token is the other one for every number."""
    say(f"[filtered] V={V} {child} {other}")
    c = _chain(V, 6)
    c["logits"][:, 0, child], c["logits"][:, 0, other] = 3.0, 1.0
    c["drafts"][:, 1] = child
    c["uniforms"][:, 0] = 0.95                                     # the child has e^2 / (1 + e^2) = 0.88
    c["uniforms"][:, 2] = [0.0, -0.0, -3.0, np.nan, 2.0 ** -24, 0.75]
    got = _run(c)
    _check(_as_counted(c), got)
    assert (got[0][:, 0] == other).all() and (got[2] == 1).all()


@pytest.mark.parametrize("seed", range(4))
def test_filtered_trees(seed):
    """Few tokens left in each row, most of them children of its node and alone in their chunks."""
    say(f"[filtered] trees {seed}")
    rng = np.random.default_rng(seed)
    B, W, V = 40, 9, 5 * CHUNK + 17
    c = _chain(V, B, W)
    c["parents"] = np.array([[-1, 0, 0, 0, 1, 1, 2, 4, 3]] * B)
    for b in range(B):
        for i in range(W):
            kept = rng.choice(6, 6, replace=False) * CHUNK + rng.integers(0, 17, 6)
            kept = np.unique(np.concatenate([kept, rng.integers(0, V, rng.integers(0, 3))]))
            c["logits"][b, i, kept] = rng.standard_normal(len(kept))
            kids = [k for k in range(W) if c["parents"][b, k] == i]
            c["drafts"][b, kids] = rng.permutation(kept)[: len(kids)]
    c["temperature"] = rng.uniform(0.4, 2.0, B).astype(np.float32)
    c["uniforms"] = rng.random((B, W + 1)).astype(np.float32)
    c["uniforms"][:, W] *= rng.random(B) < 0.3                     # the last number is 0 for most
    c["uniforms"][:, 0] = np.maximum(c["uniforms"][:, 0], np.where(rng.random(B) < 0.5, 0.97, 0)).astype(np.float32)
    got = _run(c)
    for b in range(B):
        last = got[0][b, got[2][b] - 1]
        row = c["logits"][b, got[1][b, got[2][b] - 1]]
        assert row[last] > -np.inf, f"sequence {b}: token {last} has no weight"
    _check(c, got)


def test_drawn_drafts_outside_the_filter():
    """Drawn tokens that the target's filter left out are turned down, and the last token has a weight."""
    rng = np.random.default_rng(9)
    B, W, V = 30, 3, 3 * CHUNK
    c = _chain(V, B, W)
    c["draft_logits"] = np.full((B, W, V), -np.inf, np.float32)
    for b in range(B):
        for i in range(W):
            kept = np.unique(rng.integers(0, V, 5))
            c["logits"][b, i, kept] = rng.standard_normal(len(kept))
            c["draft_logits"][b, i, np.unique(np.r_[kept[:2], rng.integers(0, V, 4)])] = rng.standard_normal()
            if i + 1 < W:
                c["drafts"][b, i + 1] = rng.choice(np.flatnonzero(c["draft_logits"][b, i] > -np.inf))
    c["uniforms"] = rng.random((B, W + 1)).astype(np.float32)
    c["uniforms"][::2, W] = 0
    got = _run(c)
    _check(c, got)
    for b in range(B):
        assert c["logits"][b, got[1][b, got[2][b] - 1], got[0][b, got[2][b] - 1]] > -np.inf
