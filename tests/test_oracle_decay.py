"""The fp64 oracles of the decayed attention and of the norm with rotation,
pinned to closed forms, to each other, to central differences and to the
oracle without a decay (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import decay as od
from oracle import norm_rope as onr

RNG = np.random.default_rng


def _case(seed, B=2, H=3, N=7, d=4):
    r = RNG(seed)
    q, k, v = (r.standard_normal((B, H, N, d)) for _ in range(3))
    return q, k, v, -np.abs(r.standard_normal(H)), r.standard_normal((B, H, d, d)), r


def test_recurrent_equals_closed_form():
    q, k, v, g, s0, _ = _case(0)
    for init in (None, s0):
        for a, b in zip(od.recurrent(q, k, v, g, init), od.masked(q, k, v, g, init)):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)


def test_no_decay_is_the_plain_oracle():
    q, k, v, g, s0, r = _case(1)
    for a, b in zip(od.recurrent(q, k, v, 0 * g, s0), oracle.recurrent(q, k, v, s0)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)
    do, ds = r.standard_normal(q.shape), r.standard_normal(s0.shape)
    for a, b in zip(od.backward(q, k, v, do, 0 * g, s0, ds), oracle.backward(q, k, v, do, s0, ds)):
        np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)


def test_full_decay_forgets_everything():
    q, k, v, g, s0, _ = _case(2)
    o, S = od.recurrent(q, k, v, np.full(3, -np.inf), s0)
    np.testing.assert_allclose(o, (q * k).sum(-1, keepdims=True) * v, rtol=1e-12)
    np.testing.assert_allclose(S, k[:, :, -1, :, None] * v[:, :, -1, None, :], rtol=1e-12)


def test_backward_against_central_differences():
    q, k, v, g, s0, r = _case(3, B=1, H=2, N=5, d=3)
    do, ds = r.standard_normal(q.shape), r.standard_normal(s0.shape)

    def loss(*x):
        o, S = od.recurrent(x[0], x[1], x[2], g, x[3])
        return (o * do).sum() + (S * ds).sum()

    args = [q, k, v, s0]
    for i, grad in enumerate(od.backward(q, k, v, do, g, s0, ds)):
        for _ in range(12):
            at = tuple(r.integers(0, n) for n in args[i].shape)
            h, vals = 1e-5, []
            for sgn in (1, -1):
                x = [a.copy() for a in args]
                x[i][at] += sgn * h
                vals.append(loss(*x))
            # the loss is multilinear: the difference quotient has no h^2 term
            assert abs((vals[0] - vals[1]) / (2 * h) - grad[at]) < 1e-8 * (1 + abs(grad[at]))


def test_varlen_and_decode_equal_the_dense_form():
    q, k, v, g, s0, _ = _case(4, B=1, N=9)
    o, S = od.recurrent(q, k, v, g, s0)
    p = [a[0].swapaxes(0, 1) for a in (q, k, v)]
    ov, Sv = od.varlen(*p, [0, 4, 4, 9], g, s0, [0, -1, -1])
    np.testing.assert_allclose(ov[:4], o[0].swapaxes(0, 1)[:4], rtol=1e-12)
    np.testing.assert_allclose(Sv[1], 0)
    o2, S2 = od.varlen(*p, [0, 4, 9], g, np.concatenate((s0, Sv[:1])), [0, 1])
    S1 = Sv[0][None]
    o3, S3 = od.recurrent(*(a[:, :, 4:] for a in (q, k, v)), g, S1)
    np.testing.assert_allclose(o2[4:], o3[0].swapaxes(0, 1), rtol=1e-12)
    np.testing.assert_allclose(S3, S, rtol=1e-11)
    state = s0
    for t in range(9):
        ot, state = od.decode(q[:, :, t], k[:, :, t], v[:, :, t], state, g)
        np.testing.assert_allclose(ot, o[:, :, t], rtol=1e-11)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_orthogonal_and_relative(interleaved):
    d, f = 8, np.array([1.0, 0.1, 0.01])
    R = onr.rotation(d, f, np.arange(6), interleaved)
    np.testing.assert_allclose(np.matmul(R, np.swapaxes(R, -1, -2)), np.broadcast_to(np.eye(d), R.shape), atol=1e-14)
    # q_m . k_n depends on m - n alone
    np.testing.assert_allclose(R[5].T @ R[2], R[4].T @ R[1], atol=1e-14)
    np.testing.assert_allclose(R[0], np.eye(d))
    np.testing.assert_allclose(R[3][6:, 6:], np.eye(2))
    a, b = (2, 3) if interleaved else (1, 4)
    np.testing.assert_allclose(R[3] @ np.eye(d)[a], np.cos(0.3) * np.eye(d)[a] + np.sin(0.3) * np.eye(d)[b], atol=1e-15)


def test_norm_rope_backward_against_central_differences():
    r = RNG(6)
    N, d = 3, 8
    x, w, dy = r.standard_normal((2, N, d)), r.standard_normal(d), r.standard_normal((2, N, d))
    R = onr.rotation(d, np.array([0.7, 0.2]), np.arange(5, 5 + N))
    dx, dw = onr.backward(dy, x, w, R, 1e-3)
    h = 1e-6
    for _ in range(20):
        at = (r.integers(2), r.integers(N), r.integers(d))
        e = np.zeros_like(x)
        e[at] = h
        num = ((onr.forward(x + e, w, R, 1e-3) - onr.forward(x - e, w, R, 1e-3)) * dy).sum() / (2 * h)
        assert abs(num - dx[at]) < 1e-7
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        num = ((onr.forward(x, w + e, R, 1e-3) - onr.forward(x, w - e, R, 1e-3)) * dy).sum() / (2 * h)
        assert abs(num - dw[i]) < 1e-7


def test_norm_of_a_row_is_its_weight():
    x = RNG(7).standard_normal((4, 16))
    y = onr.forward(x, np.ones(16), onr.rotation(16, np.ones(4), np.arange(4)), 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-12)
