"""Pins of the mixers' oracle: the rotation is a rotation, attention against a direct sum over
a permuted cache, and the recurrence against its closed form without the delta rule."""
import numpy as np

from oracle import kvfp8 as F
from oracle import mixers as M


def test_rotation_keeps_pairs_norms_and_layouts_agree():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 64)).astype(np.float32)
    ang = rng.uniform(-10, 10, 16)
    c, s = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    y = M.rotate(x, c, s, False)
    assert np.allclose(x[:, :16] ** 2 + x[:, 16:32] ** 2, y[:, :16] ** 2 + y[:, 16:32] ** 2, atol=1e-5)
    assert np.array_equal(x[:, 32:], y[:, 32:])
    z = np.concatenate([np.stack([x[:, :16], x[:, 16:32]], -1).reshape(3, 32), x[:, 32:]], 1)
    w = M.rotate(z, c, s, True)
    assert np.array_equal(w[:, 0:32:2], y[:, :16]) and np.array_equal(w[:, 1:32:2], y[:, 16:32])


def test_append_rows_and_padding():
    rng = np.random.default_rng(2)
    T, D = 5, 64
    k, v, q = (rng.standard_normal((T, h, D)).astype(np.float32) for h in (2, 2, 4))
    pool = [np.full((2, 16, 2, D), 9, np.uint8) for _ in range(2)]
    q_out = np.full((T, 4, D), 7, np.uint16)
    M.append(q, k, v, None, 0, False, None, [17, -1, 3, 32, 0], *pool, q_out, 2.0, 3.0)
    assert np.array_equal(pool[0][1, 1], F.encode(M.bf16_value(M.bf16_bits(k[0])), 2.0))
    assert np.array_equal(pool[1][0, 3], F.encode(M.bf16_value(M.bf16_bits(v[2])), 3.0))
    assert (q_out[[1, 3]] == 7).all() and (pool[0][0, 1:3] == 9).all()
    assert np.array_equal(q_out[4], M.bf16_bits(q[4]))


def test_attend_matches_direct_sum():
    rng = np.random.default_rng(3)
    q = rng.standard_normal((3, 4, 64))
    kp, vp = rng.standard_normal((2, 6, 16, 2, 64))
    table = np.array([[5, 0, 3], [1, -2, 4], [2, 2, 2]])
    out, lse, mag, _ = M.attend(q, kp, vp, table, [40, 37, 0], 48, 0.3, 21, 2)
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all()
    for b, at in ((0, list(range(19, 40))), (1, [t for t in range(16, 37) if not 16 <= t < 32])):
        for h in range(4):
            K = np.array([kp[table[b, t // 16], t % 16, h // 2] for t in at])
            V = np.array([vp[table[b, t // 16], t % 16, h // 2] for t in at])
            p = np.exp(0.3 * K @ q[b, h])
            assert np.allclose(out[b, h], p @ V / p.sum()) and np.allclose(lse[b, h], np.log(p.sum()))
            assert (mag[b, h] >= np.abs(out[b, h]) - 1e-12).all()


def test_recurrence_closed_form_and_delta():
    rng = np.random.default_rng(4)
    T, D = 9, 8
    q, k, v = rng.standard_normal((3, T, D))
    g = -rng.uniform(0, 1, T)
    S0 = rng.standard_normal((D, D))
    out, S, _ = M.recur(q, k, v, g, None, S0, 0.5)
    G = np.cumsum(g)
    for t in range(T):
        ref = np.exp(G[t]) * S0 + sum(np.exp(G[t] - G[j]) * np.outer(k[j], v[j]) for j in range(t + 1))
        assert np.allclose(out[t], 0.5 * q[t] @ ref)
    # a unit key written with beta = 1 and no decay is read back exactly
    e = k[0] / np.linalg.norm(k[0])
    _, S, _ = M.recur(q[:1], e[None], v[:1], np.zeros(1), np.ones(1), S0, 1.0)
    assert np.allclose(e @ S, v[0])
