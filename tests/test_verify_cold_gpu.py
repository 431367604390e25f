"""Verification at temperatures near 0 and at large logits: weights are e^((l - largest) / temperature), so
that the largest logits share the distribution between them, however small the temperature.  Against
oracle/drafts.py in 64 bits; tokens, paths and counts are equal where no decision lies within 2^-36 of a border."""
import numpy as np
import pytest

from gpu_util import say
from oracle import drafts as O
from test_verify_gpu import _case, _check, _run

pytestmark = pytest.mark.gpu

COLD = [1e-5, 1e-10, 3e-16, 3e-17, 3e-18, 1e-20, 1e-25, 1e-30, 1e-38, 1e-44]


def _cold(c, scale=1.0):
    B = len(COLD) * 3
    c["temperature"] = np.repeat(np.array(COLD, np.float32), 3)
    rng = np.random.default_rng(1)
    V = c["logits"].shape[2]
    for b in range(B):                              # the largest logit twice, in different chunks, here and there
        for i in range(c["logits"].shape[1]):
            if (b + i) % 2:
                row = c["logits"][b, i]
                row[rng.integers(0, V, 2)] = row.max()
    for x in (c["logits"], c["draft_logits"]):
        if x is not None:
            x += np.float32(17)
            x *= np.float32(scale)
    return c


@pytest.mark.parametrize("scale", [1.0, -1.0, 1e30])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_picked_drafts_near_temperature_0(kind, scale):
    say(f"[cold] picked {kind} {scale}")
    c = _cold(_case(3 * len(COLD), 5, 20001, seed=31, kind=kind), scale)
    _check(c, _run(c))


@pytest.mark.parametrize("scale", [1.0, 1e30])
def test_drawn_drafts_near_temperature_0(scale):
    """The chains' tokens are the draft rows' largest, of which a half are the targets' too."""
    say(f"[cold] drawn {scale}")
    c = _cold(_case(3 * len(COLD), 4, 20001, seed=32, kind="chain", sampled=True), scale)
    rng = np.random.default_rng(2)
    for b in range(3 * len(COLD)):
        for i in range(4):
            if rng.random() < 0.5:
                c["draft_logits"][b, i, c["logits"][b, i].argmax()] = 1.25 * np.abs(c["draft_logits"][b, i]).max()
            if i < 3:
                c["drafts"][b, i + 1] = c["draft_logits"][b, i].argmax()
    assert _check(c, _run(c)) > 0


def test_large_logits_at_ordinary_temperatures():
    """Logits of 1e6 and more, whose differences are a few units: only the differences count."""
    c = _case(24, 4, 9001, seed=33, kind="chain")
    c["logits"] = (np.float32(2.0 ** 20) * np.repeat([1, -1, 3], 8)[:, None, None].astype(np.float32) + np.round(8 * c["logits"]) / 8).astype(np.float32)
    _check(c, _run(c))


@pytest.mark.parametrize("sampled", [False, True])
def test_numbers_of_0_near_temperature_0(sampled):
    """0 takes the first token that has a weight: near temperature 0 the largest logits have all of it."""
    say(f"[cold] zeros {sampled}")
    c = _cold(_case(3 * len(COLD), 4, 20001, seed=34, kind="chain", sampled=sampled))
    c["temperature"] = np.minimum(c["temperature"], np.float32(1e-10))
    c["uniforms"][:, 3:] = 0
    c["uniforms"][::2] = 0
    if sampled:
        for i in range(3):
            c["drafts"][:, i + 1] = c["draft_logits"][:, i].argmax(-1)
    tokens, path, counts = _run(c)
    for b in range(len(counts)):                    # (a number of 0 and a weight of 0 lie on the border, and on its one side)
        t, p, _ = O.verify(c["logits"][b], c["drafts"][b], None, c["temperature"][b], c["uniforms"][b],
                           c["draft_logits"][b] if sampled else None)
        assert counts[b] == len(p) and list(path[b, :len(p)]) == p and list(tokens[b, :len(t)]) == t, (b, tokens[b], t)
