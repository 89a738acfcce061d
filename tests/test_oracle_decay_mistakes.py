"""Mistakes planted in the oracles of the decayed attention and of the norm with
rotation: every one is far outside the bars that the kernels are held to (CPU)."""
import numpy as np
import pytest

from oracle import decay as od
from oracle import norm_rope as onr

R = np.random.default_rng(11)
B, H, N, D = 1, 2, 40, 8
Q, K, V, DO = (R.standard_normal((B, H, N, D)) for _ in range(4))
S0, DS = (R.standard_normal((B, H, D, D)) for _ in range(2))
G = np.array([-0.05, -0.4])
LAM = np.exp(G)[:, None, None]


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def recurrence(decay_first=True, exclusive=False, lam=LAM, start=S0):
    S, o = start.copy(), np.empty_like(V)
    for t in range(N):
        kv = K[:, :, t, :, None] * V[:, :, t, None, :]
        old = S
        S = lam * S + kv if decay_first else lam * (S + kv)
        o[:, :, t] = (Q[:, :, t, None, :] @ (old if exclusive else S))[:, :, 0]
    return o, S


def test_without_a_mistake():
    for a, b in zip(recurrence(), od.recurrent(Q, K, V, G, S0)):
        assert rel(a, b) < 1e-12


@pytest.mark.parametrize("name,kw", [
    ("the new token decayed too", dict(decay_first=False)),
    ("the token itself left out", dict(exclusive=True)),
    ("the decay not exponentiated", dict(lam=1 + G[:, None, None])),
    ("the heads' decays exchanged", dict(lam=LAM[::-1])),
    ("first state left out", dict(start=0 * S0)),
    ("first state transposed", dict(start=S0.swapaxes(2, 3))),
    ("first state one decay late", dict(start=S0 / LAM)),
])
def test_forward(name, kw):
    assert rel(recurrence(**kw)[0], od.recurrent(Q, K, V, G, S0)[0]) > 2e-2, name


def gradients(lam_g=LAM, out=LAM, shift=0, transposed=False):
    G_, dk, dv = DS.copy(), np.empty_like(K), np.empty_like(V)
    for t in range(N - 1, -1, -1):
        G_ = G_ + Q[:, :, t, :, None] * DO[:, :, t, None, :]
        M = G_.swapaxes(2, 3) if transposed else G_
        dk[:, :, t] = (M @ V[:, :, t, :, None])[..., 0]
        dv[:, :, t] = (K[:, :, t, None, :] @ M)[:, :, 0]
        G_ = (lam_g if t > 0 else out) * G_
    return dk, dv, G_


def test_backward():
    _, dk, dv, ds0 = od.backward(Q, K, V, DO, G, S0, DS)
    assert max(rel(a, b) for a, b in zip(gradients(), (dk, dv, ds0))) < 1e-12
    assert rel(gradients(out=1.0)[2], ds0) > 2e-2             # dS_0 without the last decay
    assert rel(gradients(lam_g=1.0)[0], dk) > 2e-2            # no decay between tokens
    assert rel(gradients(transposed=True)[1], dv) > 2e-2
    # dq from the state before its token
    S, dq = S0.copy(), np.empty_like(Q)
    for t in range(N):
        dq[:, :, t] = (S @ DO[:, :, t, :, None])[..., 0]
        S = LAM * S + K[:, :, t, :, None] * V[:, :, t, None, :]
    assert rel(dq, od.backward(Q, K, V, DO, G, S0, DS)[0]) > 2e-2


def test_norm_and_rotation():
    x, w, dy = R.standard_normal((5, 16)), 1 + 0.3 * R.standard_normal(16), R.standard_normal((5, 16))
    f, pos, eps = np.array([1.0, 0.3, 0.1, 0.03]), np.arange(3, 8), 1e-6
    rot = onr.rotation(16, f, pos)
    y, (dx, dw) = onr.forward(x, w, rot, eps), onr.backward(dy, x, w, rot, eps)
    back = np.swapaxes(rot, -1, -2)
    turned = np.matmul(rot, x[..., None])[..., 0]
    assert rel(onr.forward(turned, w, np.eye(16)[None], eps), y) > 2e-2             # the weight after the rotation
    assert rel(onr.forward(x, w, onr.rotation(16, f, pos, True), eps), y) > 2e-2    # the other pairs
    assert rel(onr.forward(x, w, onr.rotation(16, f, pos - 1), eps), y) > 2e-2      # one position off
    assert rel(onr.forward(x, w, back, eps), y) > 2e-2                              # turned back
    mean = x / np.sqrt((x - x.mean(-1, keepdims=True)).var(-1, keepdims=True) + 0.1) * w
    assert rel(np.matmul(rot, mean[..., None])[..., 0], y) > 2e-2                   # another norm
    bdx, bdw = onr.backward(dy, x, w, back, eps)
    assert rel(bdx, dx) > 2e-2 and rel(bdw, dw) > 2e-2                              # the gradient turned the wrong way
    g = np.matmul(back, dy[..., None])[..., 0]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    assert rel(r * w * g, dx) > 2e-2                                                # without the norm's own term
    assert rel((g * x).sum(0), dw) > 2e-2                                           # of x instead of the normed x
