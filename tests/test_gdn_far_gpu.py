"""Gated delta rule prompts where they run long and at the edges of their buffers: thousands of
tokens through each of the state kernels, row bounds that are out of range (everything beside the
buffers guarded), and states beyond the 2^31st element.  Tolerances are those of test_gdn_gpu.py,
whose error grows with the square root of the tokens."""
import copy

import numpy as np
import pytest
import torch

import nvfp4_w4a4_block_act_amd as nv
from gpu_util import DEV, say
from test_gdn_gpu import Case

pytestmark = pytest.mark.gpu


def _i32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(DEV)


def _check_heads(c, key_heads, out, state, index, ends, has, scale, what=""):
    """Case.check for the value heads of some key heads (the oracle goes token by token)."""
    T, Hk, Hv, Dk, Dv = c.dims
    many = Hv // Hk
    for hk in key_heads:
        hs = slice(hk * many, (hk + 1) * many)
        one = copy.copy(c)
        one.dims = (T, 1, many, Dk, Dv)
        one.qv, one.kv, one.vv = c.qv[:, hk:hk + 1], c.kv[:, hk:hk + 1], c.vv[:, hs]
        one.g, one.beta, one.state = c.g[:, hs], None if c.beta is None else c.beta[:, hs], c.state[:, hs]
        one.check(out[:, hs], state[:, hs], index, ends, has, scale, f"{what} key head {hk}")


# 16 columns a workgroup; 32; 64 without beta (32 with it); whole heads, none of them long
@pytest.mark.parametrize("Hk,Hv,Dk,Dv,lens", [
    (1, 2, 128, 64, [4133]), (4, 8, 128, 128, [3000, 40, 1, 700, 64]), (2, 16, 64, 128, [2500, 2501, 63, 0, 129]),
    (8, 32, 64, 128, [1500, 1100, 1499, 1280, 1000, 1408, 1217, 1301])])
@pytest.mark.parametrize("delta", [True, False])
def test_thousands_of_tokens(Hk, Hv, Dk, Dv, lens, delta):
    say(f"[gdn] long {Hk}/{Hv} {Dk}x{Dv} lens={lens} delta={delta}")
    B, T = len(lens), sum(lens) + 2
    ends = np.concatenate([[0], np.cumsum(lens)])
    rng = np.random.default_rng(T)
    c = Case(T, Hk, Hv, Dk, Dv, delta, B + 1, seed=T, wide=True)
    index, has = rng.permutation(B + 1)[:B].astype(np.int32), rng.integers(0, 2, B).astype(np.int32)
    q, k, v, g, b, state = c.dev()
    out = torch.full(v.shape, 77.0, dtype=torch.bfloat16, device=DEV)
    nv.gdn_prefill(q, k, v, g, b, state, _i32(ends), has_state=_i32(has), state_index=_i32(index), out=out)
    torch.cuda.synchronize()
    _check_heads(c, sorted({0, Hk - 1}), out, state, index, ends, has, Dk ** -0.5)
    assert (out[ends[-1]:] == 77).all()


class Guarded:
    """The tensors of a call, each a part of a larger one: NaN beside the inputs, where a stray read
    would show in the results, and a pattern beside what is written."""

    def __init__(self, c, B):
        T, Hk, Hv, Dk, Dv = c.dims
        self.c, self.pairs = c, []
        q, k, v, g, b, state = c.dev()
        self.ins = [None if x is None else self.amid(x, float("nan")) for x in (q, k, v, g, b)]
        self.state = self.amid(state, 55.0)
        self.out = self.amid(torch.full(v.shape, 77.0, dtype=torch.bfloat16, device=DEV), 33.0)
        need = nv.nvfp4_gdn_prefill_workspace_bytes(T, B, Hk, Hv, Dk, Dv)
        self.ws = nv.Workspace(DEV)
        self.ws.buf = self.amid(torch.zeros(need, dtype=torch.uint8, device=DEV), 0xA5)

    def amid(self, x, fill):
        n = max(4096, 8 * (x.numel() // max(1, x.shape[0])))
        n = -(-n // 64) * 64
        whole = torch.full((x.numel() + 2 * n,), fill, dtype=x.dtype, device=DEV)
        part = whole[n:n + x.numel()]
        part.copy_(x.reshape(-1))
        self.pairs.append((whole, n, x.numel(), fill))
        return part.view(x.shape)

    def run(self, ends, **kw):
        nv.gdn_prefill(*self.ins, self.state, _i32(ends), workspace=self.ws, out=self.out, **kw)
        torch.cuda.synchronize()
        for whole, n, count, fill in self.pairs:
            for side in (whole[:n], whole[n + count:]):
                assert (torch.isnan(side).all() if fill != fill else (side == fill).all()), "a byte beside a buffer changed"


SHAPES = [(1, 1, 64, 32, 3), (2, 16, 128, 128, 5), (1, 4, 64, 128, 66), (1, 16, 128, 128, 16)]   # the last two: whole heads


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv,B", SHAPES)
def test_bounds_out_of_range_are_clamped(Hk, Hv, Dk, Dv, B, delta):
    """Bounds below 0 and beyond T, in order: the sequences are what is left of them inside [0, T]."""
    say(f"[gdn] clamped bounds {Hk}/{Hv} {Dk}x{Dv} B={B} delta={delta}")
    rng = np.random.default_rng(B)
    T = 400
    ends = np.sort(rng.integers(-60, T + 60, B + 1))
    ends[0], ends[-1] = -(1 << 31), (1 << 31) - 1
    inside = np.clip(ends, 0, T)
    c = Case(T, Hk, Hv, Dk, Dv, delta, B, seed=B)
    x = Guarded(c, B)
    x.run(ends)
    c.check(x.out, x.state, None, inside, None, Dk ** -0.5)


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv,B", SHAPES)
def test_falling_bounds_stay_inside(Hk, Hv, Dk, Dv, B, delta):
    """Bounds in any order: the results are unspecified, nothing beside the buffers is touched."""
    say(f"[gdn] falling bounds {Hk}/{Hv} {Dk}x{Dv} B={B} delta={delta}")
    T = 400
    c = Case(T, Hk, Hv, Dk, Dv, delta, B, seed=B)
    x = Guarded(c, B)
    rng = np.random.default_rng(B + 1)
    for low, high in ((0, T + 1), (-(1 << 31), (1 << 31) - 1), (-50, 450)):
        x.run(rng.integers(low, high, B + 1), has_state=_i32(rng.integers(0, 2, B)))
    x.run(([T, 0] * (B + 1))[:B + 1])


def test_states_past_two_to_the_31st_element():
    """A buffer of more than 2^31 elements: prompts and steps of its last states equal those of a
    small buffer."""
    Hk, Hv, D, far = 16, 32, 128, 4100                    # 4100 states of 2 MB, 2.15e9 elements
    c = Case(203, Hk, Hv, D, D, True, 3, seed=5)
    q, k, v, g, b, small = c.dev()
    big = torch.empty((far, Hv, D, D), device=DEV)
    assert big.numel() > 1 << 31
    where = [far - 1, 4095, 4097]
    big[where] = small
    guard = big[4096].fill_(9.0).clone()
    ends, has = _i32([0, 70, 70, 200]), _i32([1, 0, 1])
    res = []
    for state, index in ((small, [0, 1, 2]), (big, where)):
        out = nv.gdn_prefill(q[:200], k[:200], v[:200], g[:200], b[:200], state, ends, has_state=has, state_index=_i32(index))
        one = nv.gdn_step(q[200:], k[200:], v[200:], g[200:], b[200:], state, state_index=_i32(index))
        res.append((out, one, state[index]))
    torch.cuda.synchronize()
    for a, d in zip(*res):
        assert torch.equal(a, d)
    assert torch.equal(big[4096], guard)
