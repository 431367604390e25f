"""The verification of drafted tokens against oracle/drafts.py in 64 bits: tokens, paths and counts
are equal.  Probabilities and sums of both sides are binary64 (errors below 2^-40 of the total:
131072 terms of 2^-42 relative each, summed in 53 bits), so cases whose closest decision is farther
from its border than 2^-36 have one answer; the seeds are such cases, and the tests say so."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import drafts as O
from test_attn_tree_gpu import trees

pytestmark = pytest.mark.gpu


def _case(B, W, V, seed, kind="tree", sampled=False, greedy=0, spread=2.0):
    rng = np.random.default_rng(seed)
    parents = trees(B, W, seed, kind)
    if parents is not None and kind != "padded":
        parents[:, 0] = -1
    up = np.broadcast_to(np.arange(-1, W - 1), (B, W)) if parents is None else parents
    inner = np.where((up >= 0) & (up < W), up, 0)
    logits = (spread * rng.standard_normal((B, W, V))).astype(np.float32)
    temperature = rng.uniform(0.5, 1.3, B).astype(np.float32)
    temperature[:greedy] = 0
    drafts = rng.integers(0, V, (B, W))
    draft = None
    row, peak = np.arange(B)[:, None], np.log(V) + spread ** 2 / 2
    if sampled:
        peaks = rng.integers(0, V, (B, W, 6))
        np.put_along_axis(logits, peaks, (peak + rng.standard_normal((B, W, 6))).astype(np.float32), 2)
        draft = (logits + 0.4 * rng.standard_normal((B, W, V))).astype(np.float32)
        heat = np.where(temperature > 0, temperature, 1)[:, None, None]
        drawn = (draft / heat + rng.gumbel(size=(B, W, V))).argmax(-1)
        drafts = drawn[row, inner]
    else:
        logits[row, inner, drafts] = (peak + rng.standard_normal((B, W))).astype(np.float32)
        if W > 4:                                   # the same token twice among siblings, here and there
            drafts[::2, 3] = drafts[::2, 2]
    uniforms = rng.random((B, W + 1)).astype(np.float32)
    return dict(logits=logits, drafts=drafts, parents=parents, temperature=temperature, uniforms=uniforms, draft_logits=draft)


def _dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _run(c, **kw):
    d = {k: _dev(x) for k, x in c.items()}
    if d["parents"] is not None:
        d["parents"] = d["parents"].int()
    d.update(kw)
    got = nv.verify_drafts(**d)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in got]


def _check(c, got):
    tokens, path, counts = got
    B, W = c["drafts"].shape
    accepted = 0
    for b in range(B):
        t, p, margin = O.verify(c["logits"][b], c["drafts"][b], None if c["parents"] is None else c["parents"][b],
                                0.0 if c["temperature"] is None else c["temperature"][b],
                                None if c["uniforms"] is None else c["uniforms"][b],
                                None if c["draft_logits"] is None else c["draft_logits"][b])
        assert margin > 2.0 ** -36, "the seed is no test: a decision lies on a border"
        assert counts[b] == len(p) and list(path[b]) == p + [-1] * (W - len(p)), (b, path[b], p)
        assert list(tokens[b]) == t + [-1] * (W - len(t)), (b, tokens[b], t)
        accepted += max(len(p) - 1, 0)
    return accepted


@pytest.mark.parametrize("kind", ["tree", "chain", "padded"])
@pytest.mark.parametrize("B,W,V", [(1, 1, 1), (3, 1, 17), (2, 2, 8192), (5, 8, 8193), (7, 64, 1000), (4, 33, 20001), (1, 5, 131072)])
def test_picked_drafts(B, W, V, kind):
    say(f"[verify] picked B={B} W={W} V={V} {kind}")
    c = _case(B, W, V, seed=B * W + V, kind=kind, greedy=B // 3)
    _check(c, _run(c))


@pytest.mark.parametrize("kind", ["tree", "chain"])
@pytest.mark.parametrize("B,W,V", [(1, 1, 5), (6, 4, 8191), (3, 8, 24577), (9, 6, 999), (2, 5, 100003), (150, 2, 24577)])
def test_drawn_drafts(B, W, V, kind):
    say(f"[verify] drawn B={B} W={W} V={V} {kind}")
    c = _case(B, W, V, seed=B * W + V, kind=kind, sampled=True, greedy=B // 3)
    accepted = _check(c, _run(c))
    assert accepted > 0 or W == 1


def test_greedy_without_random_numbers():
    c = _case(6, 9, 5000, seed=2, greedy=6)
    c["temperature"] = c["uniforms"] = None
    for b in range(6):                                  # the first drafts of some are the largest logit's
        c["logits"][b, 0, c["drafts"][b, 1]] += 20 * (b % 2)
    c["logits"][1, 0, 4000:4003] = c["logits"][1, 0].max() + 1     # three that are equal: the lowest index
    assert _check(c, _run(c)) > 0


def test_minus_infinity_and_ties():
    """Filtered logits: -inf everywhere but a few; a row of nothing gives the token -1."""
    c = _case(4, 3, 9000, seed=4, kind="chain")
    c["logits"][:, :, 50:] = -np.inf
    c["drafts"][:, 1:] = [[7, 8]] * 4
    c["logits"][2, 1:] = -np.inf
    c["logits"][3, 0] = -np.inf
    c["uniforms"][:3, 0] = 0
    tokens, path, counts = got = _run(c)
    _check(c, got)
    assert tokens[3, 0] == -1 and counts[3] == 1
    assert counts[2] == 2 and list(tokens[2]) == [7, -1, -1]


def test_uniform_numbers_at_their_ends():
    """0 takes the first child and the first token with a weight; a number that is not below 1 counts as the
    largest below it, one that is below 0 or no number as 0: nothing leaves the vocabulary."""
    c = _case(6, 3, 9000, seed=6, kind="chain", spread=1.0)
    c["logits"][:, :, :5] = c["logits"][:, :, -5:] = -np.inf
    for b, u in enumerate([0.0, 1 - 2.0 ** -24, 1.0, np.inf, -3.0, np.nan]):
        c["uniforms"][b] = u
    tokens, _, counts = _run(c)
    again = dict(c, uniforms=np.clip(np.nan_to_num(c["uniforms"], nan=0, posinf=1), 0, np.float32(1 - 2.0 ** -24)).astype(np.float32))
    _check(again, (tokens, _run(again)[1], counts))
    assert counts[0] == 3 and tokens[0, 2] == 5 and counts[4] == counts[5] == 3
    assert ((tokens >= 5) & (tokens < 8995) | (tokens == -1)).all()


def test_no_numbers_never_fault():
    c = _case(8, 4, 9001, seed=7, sampled=True, kind="chain")
    c["logits"][0, 0, 3] = np.nan
    c["logits"][1] = np.inf
    c["logits"][2] = np.nan
    c["draft_logits"][3] = np.nan
    c["draft_logits"][4] = -np.inf
    c["temperature"][5:] = [np.nan, np.inf, 1e-38]
    tokens, path, counts = _run(c)
    assert ((tokens >= -1) & (tokens < 9001)).all() and ((counts >= 0) & (counts <= 4)).all()
    assert ((path >= -1) & (path < 4)).all()


def test_tokens_outside_the_vocabulary_are_never_accepted():
    c = _case(5, 4, 700, seed=8, kind="chain")
    c["drafts"][:, 1] = [700, -1, 1 << 40, -(1 << 62), 3]
    c["uniforms"][:, 0] = 0
    got = _run(c)
    _check(c, got)
    assert list(got[2][:4]) == [1] * 4 and got[2][4] > 1


def test_strided_logits_and_given_outputs():
    c = _case(3, 4, 5001, seed=9, sampled=True, kind="chain")
    wide = torch.full((3, 4, 5040), float("nan"), device=DEV)
    far = torch.full((3, 4, 5003), float("nan"), device=DEV)
    wide[..., :5001], far[..., :5001] = _dev(c["logits"]), _dev(c["draft_logits"])
    out = (torch.full((3, 4), 9, device=DEV), torch.full((3, 4), 9, dtype=torch.int32, device=DEV),
           torch.full((3,), 9, dtype=torch.int32, device=DEV))
    got = _run(c, logits=wide[..., :5001], draft_logits=far[..., :5001], out=out, workspace=nv.Workspace(DEV))
    _check(c, got)
    for a, b in zip(got, _run(c)):
        assert np.array_equal(a, b)


def test_first_token_has_the_targets_distribution():
    """Many sequences with the same two rows and fresh numbers: whatever was drafted, the first token's
    frequencies are p_0.  20000 draws over 12 tokens: chi squared with 11 degrees of freedom is above 45
    with a probability below 1e-5."""
    n, V, W = 20000, 12, 4
    rng = np.random.default_rng(10)
    base, other = rng.standard_normal((2, 1, W, V)).astype(np.float32)
    for sampled in (False, True):
        q = O.softmax(other[0, 0], 1.0)
        drafts = rng.choice(V, (n, W), p=q) if sampled else np.tile([0, 3, 3, 5], (n, 1))
        parents = None if sampled else np.tile(np.array([-1, 0, 0, 0], np.int32), (n, 1))
        c = dict(logits=np.repeat(base, n, 0), drafts=drafts, parents=parents, temperature=np.ones(n, np.float32),
                 uniforms=rng.random((n, W + 1)).astype(np.float32), draft_logits=np.repeat(other, n, 0) if sampled else None)
        seen = np.bincount(_run(c)[0][:, 0], minlength=V)
        want = n * O.softmax(base[0, 0], 1.0)
        assert ((seen - want) ** 2 / want).sum() < 45


def test_empty_batch():
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    tokens, path, counts = nv.verify_drafts(e(0, 3, 50), e(0, 3, dtype=torch.int64))
    assert tokens.shape == path.shape == (0, 3) and counts.shape == (0,)


def test_two_graphs_of_drawn_drafts_with_one_workspace():
    """The form whose workgroups count each other, captured twice over one workspace and replayed in turn with
    other numbers, eager calls and synchronizations between the replays: each equals an eager call."""
    ws = nv.Workspace(DEV)
    sides = []
    for seed, (B, W, V) in ((21, (3, 5, 20001)), (22, (40, 3, 9000))):
        c = {k: _dev(x) for k, x in _case(B, W, V, seed=seed, sampled=True, kind="chain", greedy=1).items()}
        c["parents"] = None
        ws.get(nv.nvfp4_verify_drafts_workspace_bytes(B, W, V, True))
        sides.append(c)
    graphs = []
    for c in sides:
        out = nv.verify_drafts(**c, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.verify_drafts(**c, workspace=ws, out=out)
        graphs.append((g, out))
    for turn in range(4):
        for c, (g, out) in zip(sides, graphs):
            c["uniforms"].copy_(_dev(np.random.default_rng(turn).random(tuple(c["uniforms"].shape)).astype(np.float32)))
            c["temperature"][-1] = 0.0 if turn % 2 else 0.9
            for o in out:
                o.fill_(7)
            g.replay()
            want = nv.verify_drafts(**c)
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), f"turn {turn}"
