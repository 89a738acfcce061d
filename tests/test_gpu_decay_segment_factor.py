"""The factor exp(len g) by which a state passes a segment, repeated over a
hundred segments: without keys the last state is exp(N g) S_0, so an error of the
factor is not covered by the segments' sums.

Tolerance.  A state passes 100 segments and the chunk or two of the last one:
at most 104 products, each rounded by at most 2^-24 of itself, with factors near
0.55, so that the mantissas have nothing to do with each other: sqrt(104) 2^-24 =
6.1e-7 in the 2-norm.  (A second rounding of a product's small part is 2^-48.)  One
fp32 factor is off by 5e-8 or more here: 5e-6 after 100 segments.
"""
import math

import numpy as np
import pytest
import torch

import synth
from tests.parity import rel_per_unit, to64

pytestmark = pytest.mark.gpu
TOL = math.sqrt(104) * 2.0 ** -24
P = 100


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


def decays(seg_len, H=2):
    """log decays whose exp(seg_len g), near 0.55, lies furthest from an fp32 value."""
    g = np.arange(4000, dtype=np.float64) * 1e-6 / seg_len + math.log(0.55) / seg_len
    g = g.astype(np.float32)
    f = np.exp(g.astype(np.float64) * seg_len)
    off = np.abs(f.astype(np.float32) / f - 1)
    best = np.argsort(off)[-H:]
    assert off[best].min() > 5e-8
    return torch.from_numpy(g[best])


def states(H, d):
    return synth.outer_product_state(H, d, d, [64] * H, seed=3).view(1, H, d, d)


@pytest.mark.parametrize("dtype,d,seg_len", [("fp32", 64, 64), ("fp32", 128, 64), ("bf16", 128, 128), ("bf16", 64, 128)])
def test_dense_both_ways(la, monkeypatch, dtype, d, seg_len):
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", str(P))
    H, N = 2, P * seg_len
    g = decays(seg_len)
    s0 = states(H, d)
    want = to64(s0) * np.exp(to64(g) * N)[:, None, None]
    q, k, v = (t.cuda() for t in synth.dense(1, H, N, d, dtype, seed=4))
    zero = torch.zeros_like(k)
    _, S = la.prefill(q, zero, v, s0.cuda(), log_decay=g.cuda())
    assert rel_per_unit(S.cpu(), want, 2).max() <= TOL
    # the state's gradient on its way back, without queries
    *_, ds0 = la.prefill_backward(zero, k, v, v, None, s0.cuda(), log_decay=g.cuda())
    assert rel_per_unit(ds0.cpu(), want, 2).max() <= TOL


@pytest.mark.parametrize("dtype,d", [("fp32", 64), ("bf16", 128)])
def test_packed(la, monkeypatch, dtype, d):
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", str(P))
    H, lens = 2, [P * 128, 389]
    g, pool = decays(128), states(2, d)
    cu = synth.cu_seqlens(lens).cuda()
    q, k, v = (t.cuda() for t in synth.qkv((sum(lens), H, d), d, dtype, seed=5))
    _, S = la.prefill_varlen(q, torch.zeros_like(k), v, cu, pool.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"),
                             log_decay=g.cuda())
    for n, N in enumerate(lens):
        want = to64(pool) * np.exp(to64(g) * N)[:, None, None]
        assert rel_per_unit(S[n:n + 1].cpu(), want, 2).max() <= TOL
