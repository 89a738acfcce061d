"""Infinite values in the decayed attention: a state that holds an infinity (an
fp16 one overflows at 65504) keeps it, as the recurrence says and as the calls
without a decay do.  An infinite key or value makes the state entries that it
reaches infinite, or NaN on the tensor cores, and nothing else."""
import numpy as np
import pytest
import torch

import synth
from oracle import decay as od
from tests.parity import to64

pytestmark = pytest.mark.gpu
INF = float("inf")
G = torch.tensor([0.0, -1e-3, -0.02])  # exp(n g) stays far above the smallest fp32 value at the lengths here


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def same_kind(got, ref):
    """Finite, NaN, +inf or -inf at the same places."""
    got, ref = to64(got), to64(ref)
    for f in (np.isnan, np.isposinf, np.isneginf):
        np.testing.assert_array_equal(f(got), f(ref))


def finite_close(got, ref, tol):
    got, ref = to64(got), to64(ref)
    ok = np.isfinite(ref)
    assert np.linalg.norm(got[ok] - ref[ok]) <= tol * np.linalg.norm(ref[ok])


def state(H, d):
    S = synth.outer_product_state(H, d, d, [64] * H, seed=1).view(1, H, d, d)
    S[:, :, 3, 5], S[:, :, d - 1, 0] = INF, -INF
    return S


@pytest.mark.parametrize("sdt", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_keeps_an_infinite_state(la, sdt, d):
    q, k, v = synth.qkv((1, 3, d), d, "bf16", seed=2)
    S = state(3, d).to(getattr(torch, sdt)).cuda()
    plain = S.clone()
    with np.errstate(invalid="ignore"):
        ro, rS = od.decode(q, k, v, S.cpu(), G)
    o = la.decode_step(*cuda(q, k, v), S, log_decay=G.cuda())
    po = la.decode_step(*cuda(q, k, v), plain)
    same_kind(S.float().cpu(), rS)
    same_kind(o.cpu(), ro)
    assert torch.equal(S[:, 0], plain[:, 0]) and torch.equal(o[:, 0], po[:, 0])  # head 0 has no decay


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("segments", ["1", "3"])
def test_prefill_keeps_an_infinite_state(la, monkeypatch, dtype, d, segments):
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", segments)
    q, k, v = synth.dense(1, 3, 500, d, dtype, seed=3)
    s0 = state(3, d)
    o, S = la.prefill(*cuda(q, k, v, s0), log_decay=G.cuda())
    with np.errstate(invalid="ignore"):
        ro, rS = od.recurrent(q, k, v, G, s0)
    same_kind(S.cpu(), rS)
    finite_close(S.cpu(), rS, 5e-6)
    same_kind(o.cpu(), ro)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64)])
def test_packed_prefill_keeps_an_infinite_state(la, dtype, d):
    lens = [200, 0, 1, 300]
    cu = synth.cu_seqlens(lens)
    q, k, v = synth.qkv((int(cu[-1]), 3, d), d, dtype, seed=4)
    pool, idx = state(3, d), torch.tensor([0, 0, -1, 0], dtype=torch.int32)
    o, S = la.prefill_varlen(*cuda(q, k, v, cu, pool, idx), log_decay=G.cuda())
    with np.errstate(invalid="ignore"):
        ro, rS = od.varlen(q, k, v, cu, G, pool, idx)
    same_kind(S.cpu(), rS)
    same_kind(o.cpu(), ro)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64)])
def test_backward_keeps_infinite_state_gradients(la, dtype, d):
    q, k, v = synth.dense(1, 3, 300, d, dtype, seed=5)
    do = synth.dense(1, 3, 300, d, dtype, seed=6)[2]
    ds = state(3, d)
    got = la.prefill_backward(*cuda(q, k, v, do, None, ds), log_decay=G.cuda())
    with np.errstate(invalid="ignore"):
        ref = od.backward(q, k, v, do, G, None, ds)
    for a, b in zip(got, ref):
        same_kind(a.cpu(), b)


def kind_by_path(got, ref, dtype):
    """The recurrence's kind on the FFMA kernel; on the tensor cores NaN may stand for an infinity."""
    if dtype == "fp32":
        same_kind(got, ref)
    else:
        np.testing.assert_array_equal(np.isfinite(to64(got)), np.isfinite(to64(ref)))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
@pytest.mark.parametrize("segments", ["1", "3"])
@pytest.mark.parametrize("at", [150, 255, 390])
def test_an_infinite_value(la, monkeypatch, dtype, d, segments, at):
    """Only the value's column is touched, in the chunk of its token and later ones."""
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", segments)
    q, k, v = synth.dense(1, 3, 400, d, dtype, seed=7)
    v[:, :, at, 7] = INF
    o, S = la.prefill(*cuda(q, k, v), log_decay=G.cuda())
    with np.errstate(invalid="ignore"):
        ro, rS = od.recurrent(q, k, v, G)
    kind_by_path(S.cpu(), rS, dtype)
    finite_close(S.cpu(), rS, 5e-6)
    o, ro = to64(o.cpu()), to64(ro)
    rest, first = np.arange(d) != 7, at // 128 * 128
    for a, b in ((o[..., rest], ro[..., rest]), (o[:, :, :first], ro[:, :, :first])):
        assert np.isfinite(a).all() and np.linalg.norm(a - b) <= 5e-3 * np.linalg.norm(b)
    # from the token on the column is lost
    assert not np.isfinite(o[:, :, at:, 7]).any()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
@pytest.mark.parametrize("segments", ["1", "3"])
@pytest.mark.parametrize("at", [150, 255, 390])
def test_an_infinite_key(la, monkeypatch, dtype, d, segments, at):
    """Every output from its token on is lost, those before it are right; of the state one row is lost."""
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", segments)
    q, k, v = synth.dense(1, 3, 400, d, dtype, seed=8)
    k[:, :, at, 7] = -INF
    o, S = la.prefill(*cuda(q, k, v), log_decay=G.cuda())
    with np.errstate(invalid="ignore"):
        ro, rS = od.recurrent(q, k, v, G)
    kind_by_path(S.cpu(), rS, dtype)
    finite_close(S.cpu(), rS, 5e-6)
    kind_by_path(o.cpu(), ro, dtype)
    finite_close(o.cpu(), ro, 5e-3)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
def test_an_infinite_output_gradient(la, dtype, d):
    q, k, v = synth.dense(1, 3, 300, d, dtype, seed=9)
    do = synth.dense(1, 3, 300, d, dtype, seed=10)[2]
    do[:, :, 140, 7] = INF
    _, dk, dv, ds0 = la.prefill_backward(*cuda(q, k, v, do), log_decay=G.cuda())
    with np.errstate(invalid="ignore"):
        _, rdk, rdv, rds0 = od.backward(q, k, v, do, G)
    kind_by_path(ds0.cpu(), rds0, dtype)
    kind_by_path(dk.cpu(), rdk, dtype)
    kind_by_path(dv[:, :, :128].cpu(), rdv[:, :, :128], dtype)


def test_an_infinite_value_in_a_packed_batch(la):
    """Only the sequence that holds it is touched."""
    d, lens = 128, [200, 70, 300]
    cu = synth.cu_seqlens(lens)
    q, k, v = synth.qkv((int(cu[-1]), 3, d), d, "bf16", seed=11)
    v[250, :, 7] = INF
    o, S = la.prefill_varlen(*cuda(q, k, v, cu), log_decay=G.cuda())
    with np.errstate(invalid="ignore"):
        ro, rS = od.varlen(q, k, v, cu, G)
    kind_by_path(S.cpu(), rS, "bf16")
    finite_close(S.cpu(), rS, 5e-6)
    for part in (slice(0, 200), slice(270, None)):
        finite_close(o[part].cpu(), ro[part], 5e-3)
        assert torch.isfinite(o[part]).all()
