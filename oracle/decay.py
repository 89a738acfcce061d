"""fp64 oracle of the linear attention with a decay per head — TEST INFRASTRUCTURE ONLY.

Token by token, as the recurrence is written (numpy, float64, all units at
once; it shares no code with the CUDA library):

    S_t = exp(g_h) S_{t-1} + k_t v_t^T,   o_t = q_t S_t          (recurrent)
    G_t = q_t^T do_t + exp(g_h) G_{t+1},  G_N = q_N^T do_N + dS_N,
    dq_t = do_t S_t^T, dk_t = G_t v_t, dv_t = G_t^T k_t, dS_0 = exp(g_h) G_1   (backward)

``masked`` is the same in one product over all token pairs, for the pins.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        a = a.detach().to("cpu").double().numpy()
    return np.asarray(a, dtype=np.float64)


def _lam(log_decay):
    return np.exp(_f64(log_decay))[:, None, None]


def recurrent(q, k, v, log_decay, s0=None):
    """q, k, v [B, H, N, d], log_decay [H], s0 [B, H, d, d] or None -> (o, S_N)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, N, d = q.shape
    lam = _lam(log_decay)
    S = np.zeros((B, H, d, v.shape[-1])) if s0 is None else _f64(s0).copy()
    o = np.empty(v.shape)
    for t in range(N):
        S = lam * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        o[:, :, t] = np.matmul(q[:, :, t, None, :], S)[:, :, 0]
    return o, S


def masked(q, k, v, log_decay, s0=None):
    """The closed form: o_t = sum_{s <= t} e^(g (t - s)) (q_t . k_s) v_s + e^(g t) q_t S_0, t = 1 .. N."""
    q, k, v, g = _f64(q), _f64(k), _f64(v), _f64(log_decay)
    N = q.shape[2]
    t = np.arange(1, N + 1)
    gap = t[:, None] - t[None, :]
    with np.errstate(invalid="ignore"):
        w = np.where(gap > 0, np.exp(g[:, None, None] * np.maximum(gap, 1)), (gap == 0) * 1.0)
        last = np.where(N - t > 0, np.exp(g[:, None] * np.maximum(N - t, 1)), 1.0)
        first = np.exp(g[:, None] * t)
        all_n = np.exp(g * N) if N else np.ones_like(g)
    o = np.matmul(np.matmul(q, k.swapaxes(2, 3)) * w, v)
    S = np.matmul((k * last[:, :, None]).swapaxes(2, 3), v)
    if s0 is not None:
        s0 = _f64(s0)
        o = o + first[:, :, None] * np.matmul(q, s0)
        S = S + all_n[:, None, None] * s0
    return o, S


def varlen(q, k, v, cu_seqlens, log_decay, pool=None, init_idx=None):
    """Packed [T, H, d]; rows behind the last sequence are zero here."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    cu = [int(x) for x in cu_seqlens]
    H, d = q.shape[1:]
    o, states = np.zeros(v.shape), []
    for n in range(len(cu) - 1):
        i = -1 if init_idx is None else int(init_idx[n])
        s0 = None if pool is None or i < 0 else _f64(pool[i])[None]
        x = [a[cu[n]:cu[n + 1]].swapaxes(0, 1)[None] for a in (q, k, v)]
        on, S = recurrent(*x, log_decay, s0)
        o[cu[n]:cu[n + 1]] = on[0].swapaxes(0, 1)
        states.append(S[0])
    return o, np.stack(states) if states else np.zeros((0, H, d, d))


def decode(q, k, v, S, log_decay):
    """One token, q, k, v [B, H, d]: (o, S_new) before any rounding of the stored state."""
    q, k, v, S = _f64(q), _f64(k), _f64(v), _f64(S)
    S = _lam(log_decay) * S + k[..., :, None] * v[..., None, :]
    return np.matmul(q[..., None, :], S)[..., 0, :], S


def backward(q, k, v, do, log_decay, s0=None, ds_n=None):
    """(dq, dk, dv, dS_0)."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    B, H, N, d = q.shape
    lam = _lam(log_decay)
    S = np.zeros((B, H, d, d)) if s0 is None else _f64(s0).copy()
    dq, dk, dv = np.empty_like(q), np.empty_like(k), np.empty_like(v)
    for t in range(N):
        S = lam * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        dq[:, :, t] = np.matmul(S, do[:, :, t, :, None])[..., 0]
    G = np.zeros((B, H, d, d)) if ds_n is None else _f64(ds_n).copy()  # dL/dS_t, without token t's own term
    for t in range(N - 1, -1, -1):
        G = G + q[:, :, t, :, None] * do[:, :, t, None, :]
        dk[:, :, t] = np.matmul(G, v[:, :, t, :, None])[..., 0]
        dv[:, :, t] = np.matmul(k[:, :, t, None, :], G)[:, :, 0]
        G = lam * G
    return dq, dk, dv, G
