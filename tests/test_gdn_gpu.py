"""GPU parity of the gated delta rule, single tokens and prompts, against the token-by-token
recurrence of oracle/mixers.py in 64 bits.

Tolerance.  Keys have unit length, beta is in (0, 1) and decays are at most 1, so a token's map
of the state has norm at most 1 and the errors of the tokens add: each is a few binary32
roundings of sums of k_dim products, independent of one another, of norm about 2^-24 of the
largest state L on the way (||v|| included).  After n tokens ||dS|| is about sqrt(n) 2^-24 L; the
tests allow 8 sqrt(n + 8) 2^-24 L, far below one rounding to bf16 (2^-9).  An output is off by
the bf16 rounding (2^-8 of itself), by dS, and by at most 2^-14 scale ||q|| L for operands that
enter its two products to 16 bits or more."""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from oracle import mixers as M

pytestmark = pytest.mark.gpu


def _bf16(x):
    b = M.bf16_bits(np.asarray(x, np.float32))
    return M.bf16_value(b).astype(np.float64), torch.from_numpy(b.view(np.int16)).to(DEV).view(torch.bfloat16)


class Case:
    def __init__(self, T, Hk, Hv, Dk, Dv, delta, states, seed=0, rate=0.3, wide=False):
        rng = np.random.default_rng(seed)
        unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
        self.dims = (T, Hk, Hv, Dk, Dv)
        self.qv, self.q = _bf16(unit(rng.standard_normal((T, Hk, Dk)) + 0.3))
        self.kv, self.k = _bf16(unit(rng.standard_normal((T, Hk, Dk)) + 0.3))     # keys with something in common
        self.vv, self.v = _bf16(rng.standard_normal((T, Hv, Dv)))
        self.g = (-rate * rng.exponential(1.0, (T, Hv)) * rng.choice([0.01, 1.0, 20.0], (1, Hv))).astype(np.float32)
        self.beta = rng.uniform(0.01, 0.99, (T, Hv)).astype(np.float32) if delta else None
        self.state = rng.standard_normal((states, Hv, Dk, Dv)).astype(np.float32)
        self.wide = wide

    def dev(self):
        to = lambda a: None if a is None else torch.from_numpy(a.copy()).to(DEV)  # noqa: E731
        q, k, v, g, b = self.q, self.k, self.v, to(self.g), to(self.beta)
        T, Hk, Hv, Dk, Dv = self.dims
        if self.wide:                                     # columns of one fused tensor
            f = torch.cat([q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)], 1)
            q, k, v = (p.view(T, -1, d) for p, d in zip(f.split([Hk * Dk, Hk * Dk, Hv * Dv], 1), (Dk, Dk, Dv)))
            if b is not None:
                gb = torch.cat([g, b], 1)
                g, b = gb[:, :Hv], gb[:, Hv:]
        return q, k, v, g, b, to(self.state)

    def check(self, out, state, index, ends, has, scale, what=""):
        T, Hk, Hv, Dk, Dv = self.dims
        f64 = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
        ref, S, L = M.gdn(self.qv, self.kv, self.vv, f64(self.g), f64(self.beta), self.state, index, ends, has, scale)
        out, state = out.cpu().double().numpy(), state.cpu().double().numpy()
        for b in range(len(ends) - 1):
            n, slot = ends[b + 1] - ends[b], b if index is None else index[b]
            if slot < 0 or slot >= len(S):
                continue
            for h in range(Hv):
                vn = np.linalg.norm(self.vv[ends[b]:ends[b + 1], h], axis=-1).max() if n else 0.0
                big = L[slot, h] + vn
                tol = 8 * np.sqrt(n + 8) * 2.0 ** -24 * big
                d = np.linalg.norm(state[slot, h] - S[slot, h])
                assert d <= tol, f"{what}: state of sequence {b} head {h} off by {d:.2e}, tolerance {tol:.2e}"
                o, r = out[ends[b]:ends[b + 1], h], ref[ends[b]:ends[b + 1], h]
                qn = np.linalg.norm(self.qv[ends[b]:ends[b + 1], h // (Hv // Hk)], axis=-1, keepdims=True)
                to = 2.0 ** -8 * np.abs(r) + scale * qn * (tol + 2.0 ** -14 * big) + 1e-30
                assert (np.abs(o - r) <= to).all(), f"{what}: outputs of sequence {b} head {h}"
        kept = np.ones(len(S), bool)
        kept[[x for x in (range(len(ends) - 1) if index is None else index) if 0 <= x < len(S)]] = False
        assert np.array_equal(state[kept], self.state[kept].astype(np.float64)), f"{what}: other states changed"


@pytest.mark.parametrize("batch", [40, 140])
def test_step_of_large_states(batch):
    """States of 80 MB (hinted loads) and 280 MB (stores too): the first and last sequences
    against the oracle, and all of them against the same tokens one sequence at a time."""
    g = torch.Generator(DEV).manual_seed(batch)
    c = Case(2, 16, 32, 128, 128, True, 2, seed=batch)
    small = c.dev()
    rep = [x.repeat_interleave(batch // 2, 0).contiguous() for x in small]
    order = torch.randperm(batch, device=DEV, generator=g).int()
    state = torch.empty_like(rep[5])
    state[order.long()] = rep[5]
    out = nv.gdn_step(*rep[:5], state, state_index=order)
    one = nv.gdn_step(*small)
    torch.cuda.synchronize()
    c.check(one, small[5], None, [0, 1, 2], np.ones(2), 128 ** -0.5)
    # the sums of the rows are taken in another order than for two sequences: a few roundings apart
    want = small[5].repeat_interleave(batch // 2, 0)
    d = (state[order.long()] - want).flatten(1).norm(dim=1)
    assert (d <= 16 * 2.0 ** -24 * want.flatten(1).norm(dim=1)).all()
    for b in range(batch):
        assert torch.equal(out[b], out[b // (batch // 2) * (batch // 2)])
    d = (out.double() - one.repeat_interleave(batch // 2, 0).double()).abs()
    assert (d <= 2.0 ** -7 * out.double().abs() + 1e-5).all()


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 16, 32, 128, 128), (5, 2, 6, 64, 32), (33, 4, 4, 128, 64), (3, 1, 2, 128, 1024),
                                           (7, 2, 2, 64, 96), (130, 2, 4, 64, 128), (70, 8, 8, 128, 256)])
def test_step(B, Hk, Hv, Dk, Dv, delta):
    say(f"[gdn] step B={B} heads={Hk}/{Hv} dims={Dk}x{Dv} delta={delta}")
    c = Case(B, Hk, Hv, Dk, Dv, delta, B + 2, seed=B + Dv, wide=B % 2 == 1)
    index = np.random.default_rng(B).permutation(B + 2)[:B].astype(np.int32)
    if B > 4:
        index[1], index[3] = -1, B + 2
    q, k, v, g, b, state = c.dev()
    out = torch.full(v.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    got = nv.gdn_step(q, k, v, g, b, state, state_index=torch.from_numpy(index).to(DEV), scale=0.3, out=out)
    torch.cuda.synchronize()
    assert got is out
    c.check(out, state, index, list(range(B + 1)), np.ones(B), 0.3)
    if B > 4:
        assert (out[[1, 3]] == 77).all()


PROMPTS = [[1], [64], [65], [63, 0, 1], [17, 128, 5, 200, 0], [300], [0, 0], [257, 66]]


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("lens", PROMPTS)
def test_prompt_lengths(lens, delta):
    say(f"[gdn] prompt lens={lens} delta={delta}")
    B, T = len(lens), sum(lens) + 3                        # three rows belong to no sequence
    c = Case(T, 2, 4, 128, 64, delta, B + 1, seed=T, wide=True)
    ends = np.concatenate([[0], np.cumsum(lens)])
    index = np.random.default_rng(T).permutation(B + 1)[:B].astype(np.int32)
    has = (np.arange(B) % 2 == 0).astype(np.int32)
    q, k, v, g, b, state = c.dev()
    out = torch.full(v.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    nv.gdn_prefill(q, k, v, g, b, state, to(ends), has_state=to(has), state_index=to(index), out=out)
    torch.cuda.synchronize()
    c.check(out, state, index, ends, has, 128 ** -0.5)
    assert (out[ends[-1]:] == 77).all()


@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 1, 64, 32), (2, 6, 64, 96), (1, 2, 128, 256), (3, 3, 64, 128), (1, 1, 128, 1024)])
@pytest.mark.parametrize("delta", [True, False])
def test_prompt_layouts(Hk, Hv, Dk, Dv, delta):
    lens = [70, 130]
    c = Case(200, Hk, Hv, Dk, Dv, delta, 2, seed=Dv)
    q, k, v, g, b, state = c.dev()
    out = nv.gdn_prefill(q, k, v, g, b, state, torch.tensor([0, 70, 200], dtype=torch.int32, device=DEV), scale=0.5)
    torch.cuda.synchronize()
    c.check(out, state, None, [0, 70, 200], None, 0.5)
    assert sum(lens) == 200


# Many heads: workgroups of 32 columns, and of 64 without beta; batches around the 64 sequences
# that are put in order by length.
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(3, 2, 16, 64, 128), (3, 4, 16, 128, 128), (5, 8, 16, 128, 128), (5, 4, 16, 64, 128),
                                           (6, 2, 12, 64, 96), (64, 1, 6, 64, 64), (65, 1, 5, 128, 64), (80, 2, 4, 128, 192)])
@pytest.mark.parametrize("delta", [True, False])
def test_prompts_of_many_heads(B, Hk, Hv, Dk, Dv, delta):
    say(f"[gdn] prompts B={B} heads={Hk}/{Hv} dims={Dk}x{Dv} delta={delta}")
    rng = np.random.default_rng(B + Dv)
    lens = rng.integers(0, 9 if B > 10 else 150, B)
    lens[B // 2] = 130
    ends = np.concatenate([[0], np.cumsum(lens)])
    T = int(ends[-1]) + 2
    c = Case(T, Hk, Hv, Dk, Dv, delta, B + 2, seed=T)
    index = rng.permutation(B + 2)[:B].astype(np.int32)
    index[1] = -1                                          # a padded row
    has = rng.integers(0, 2, B).astype(np.int32)
    q, k, v, g, b, state = c.dev()
    out = torch.full(v.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    nv.gdn_prefill(q, k, v, g, b, state, to(ends), has_state=to(has), state_index=to(index), out=out)
    torch.cuda.synchronize()
    c.check(out, state, index, ends, has, 128 ** -0.5 if Dk == 128 else 0.125)
    assert (out[ends[-1]:] == 77).all() and (out[ends[1]:ends[2]] == 77).all()


# Heads enough for a workgroup each: some sequences long beside the others (those go another
# way), none, all empty but one, more than 64, two slabs of 128 columns, the last rows partial.
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv,lens", [
    (2, 16, 128, 128, [64] * 9 + [65] * 9), (4, 16, 64, 128, [1, 63, 128, 0, 200, 7] * 3), (2, 16, 128, 256, [70] * 8 + [0]),
    (1, 4, 64, 128, [3] * 66 + [0, 1, 250, 2]), (1, 32, 64, 128, [0] * 7 + [140]), (2, 4, 128, 128, [300] + [5] * 68 + [66])])
def test_prompts_by_whole_heads(Hk, Hv, Dk, Dv, lens, delta):
    say(f"[gdn] whole heads {Hk}/{Hv} {Dk}x{Dv} lens={lens[:4]}.. delta={delta}")
    B, T = len(lens), sum(lens) + 1
    assert B * Hv * (Dv // 128) >= 256
    ends = np.concatenate([[0], np.cumsum(lens)])
    rng = np.random.default_rng(T)
    c = Case(T, Hk, Hv, Dk, Dv, delta, B + 1, seed=T, wide=True)
    index, has = rng.permutation(B + 1)[:B].astype(np.int32), rng.integers(0, 2, B).astype(np.int32)
    index[2] = B + 1                                       # a padded row
    q, k, v, g, b, state = c.dev()
    out = torch.full(v.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    to = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
    nv.gdn_prefill(q, k, v, g, b, state, to(ends), has_state=to(has), state_index=to(index), out=out)
    torch.cuda.synchronize()
    c.check(out, state, index, ends, has, Dk ** -0.5)
    assert (out[ends[-1]:] == 77).all() and (out[ends[2]:ends[3]] == 77).all()


def test_one_state_twice_disturbs_no_other():
    """Two sequences of one state: its contents are unspecified, every other state and output is right."""
    c = Case(90, 2, 4, 64, 32, True, 4, seed=14)
    q, k, v, g, b, state = c.dev()
    to = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    out = nv.gdn_prefill(q, k, v, g, b, state, to([0, 40, 70, 90]), state_index=to([1, 1, 3]))
    alone_state = torch.from_numpy(c.state).to(DEV)
    alone = nv.gdn_prefill(q[70:], k[70:], v[70:], g[70:], b[70:], alone_state, to([0, 20]), state_index=to([3]))
    torch.cuda.synchronize()
    assert torch.equal(out[70:], alone) and torch.equal(state[[0, 2, 3]], alone_state[[0, 2, 3]])


@pytest.mark.parametrize("rate", [0.0, 0.002, 5.0, 1000.0])
def test_prompt_decays(rate):
    """No decay at all, slow ones, and ones that underflow within a chunk; some of -inf."""
    c = Case(190, 2, 2, 128, 32, True, 1, seed=int(rate), rate=rate)
    if rate == 5.0:
        c.g[[10, 64, 127, 128], 1] = -np.inf
    q, k, v, g, b, state = c.dev()
    has = torch.ones(1, dtype=torch.int32, device=DEV)
    out = nv.gdn_prefill(q, k, v, g, b, state, torch.tensor([0, 190], dtype=torch.int32, device=DEV), has_state=has)
    torch.cuda.synchronize()
    c.check(out, state, None, [0, 190], np.ones(1), 128 ** -0.5)


def test_repeated_keys_and_full_writes():
    """beta = 1 and one key throughout: each write replaces the last, the hardest chunk to solve."""
    c = Case(150, 1, 2, 128, 64, True, 1, seed=1, rate=0.01)
    c.kv[:], c.k[:] = c.kv[:1], c.k[:1].clone()
    c.kv /= np.linalg.norm(c.kv[0, 0])                    # exactly unit for the oracle's bound ...
    c.kv, c.k = _bf16(c.kv)                               # ... up to the rounding both sides see
    c.beta[:] = 1.0
    q, k, v, g, b, state = c.dev()
    out = nv.gdn_prefill(q, k, v, g, b, state, torch.tensor([0, 150], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    c.check(out, state, None, [0, 150], None, 128 ** -0.5)


def test_prompt_then_steps_equals_one_prompt():
    """A prompt in two calls and single tokens after it, against the oracle over all of it."""
    T, cut = 140, 130
    c = Case(T, 2, 4, 128, 128, True, 1, seed=11)
    q, k, v, g, b, state = c.dev()
    ends = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    has = torch.ones(1, dtype=torch.int32, device=DEV)
    out = torch.empty(v.shape, dtype=torch.bfloat16, device=DEV)
    nv.gdn_prefill(q[:70], k[:70], v[:70], g[:70], b[:70], state, ends(70), out=out[:70])
    nv.gdn_prefill(q[70:cut], k[70:cut], v[70:cut], g[70:cut], b[70:cut], state, ends(cut - 70), has_state=has,
                   out=out[70:cut])
    for t in range(cut, T):
        r = slice(t, t + 1)
        nv.gdn_step(q[r], k[r], v[r], g[r], b[r], state, out=out[r])
    torch.cuda.synchronize()
    c.check(out, state, None, [0, T], None, 128 ** -0.5)


def test_bad_row_bounds_stay_inside():
    """Row bounds beyond T or falling are clamped: nothing outside is touched."""
    c = Case(100, 1, 1, 64, 32, True, 3, seed=12)
    q, k, v, g, b, state = c.dev()
    out = torch.full(v.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    nv.gdn_prefill(q, k, v, g, b, state, torch.tensor([-5, 40, 30, 1 << 30], dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    assert torch.isfinite(state).all() and torch.isfinite(out.float()).all()


def test_refusals():
    c = Case(8, 2, 4, 128, 64, True, 8, seed=13)
    q, k, v, g, b, state = c.dev()
    ok = (q, k, v, g, b, state)
    for i, wrong in ((0, q.float()), (1, k[:, :1]), (2, v[:7]), (3, g.double()), (4, b[:, :2]), (5, state.bfloat16()),
                     (5, state[:, :, :, :32])):
        with pytest.raises(AssertionError):
            nv.gdn_step(*ok[:i], wrong, *ok[i + 1:])
    with pytest.raises(AssertionError):
        nv.gdn_step(*ok, state_index=torch.zeros(8, dtype=torch.int64, device=DEV))
    with pytest.raises(nv.NVFP4Error):
        nv.gdn_step(*ok[:5], state[:7])
    with pytest.raises(AssertionError):
        nv.gdn_prefill(*ok, torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(nv.NVFP4Error):
        nv.gdn_prefill(*ok, torch.zeros(3, dtype=torch.int32, device=DEV), scale=float("inf"))
