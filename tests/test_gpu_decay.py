"""Linear attention with a decay per head (``log_decay``) against the fp64
oracle: prefill, ragged prefill, decode and backward.

Tolerances.  Outputs: the bars of tests/parity.py (bf16: three roundings of
half a step, 2^-8 at most and about 1.6e-3 in the 2-norm each: scores, state
operand, output; fp32: 1e-4).  States are fp32: a state is a sum of at most n
rounded products, each rounding at most 2^-24 of its partial sum, so in the
2-norm the error stays below sqrt(n) 2^-24 for independent roundings; with n <=
4096 here, 4e-6, and STATE takes 5e-6.
"""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import decay as od
from tests.parity import assert_guard_intact, assert_out, assert_state, assert_varlen_out, guarded, rel_per_unit, to64

pytestmark = pytest.mark.gpu
STATE = 5e-6


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


def ladder(H, kind="ladder"):
    """log decays of H heads: a geometric ladder of slopes; heads of no, slow, strong and full decay."""
    if kind == "ladder":
        return -torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
    mix = [0.0, -1e-6, -1e-3, -0.1, -1.0, -3.0, -20.0, -300.0, -math.inf]
    return torch.tensor([mix[(3 * h) % len(mix)] if H < len(mix) else mix[h % len(mix)] for h in range(H)])


def states(B, H, d, seed):
    return synth.outer_product_state(B * H, d, d, [64] * (B * H), seed=seed).view(B, H, d, d)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def run_prefill(la, q, k, v, g, s0, **kw):
    B, H, N, d = q.shape
    o, o_full = guarded(v.shape, q.dtype)
    s, s_full = guarded((B, H, d, d), torch.float32)
    la.prefill(*cuda(q, k, v, s0), out=o, s_out=s, log_decay=g.cuda(), **kw)
    torch.cuda.synchronize()
    assert la.device_status() == 0
    assert_guard_intact(o_full, o.numel())
    assert_guard_intact(s_full, s.numel())
    return o.cpu(), s.cpu()


KINDS = [("bf16", 128, 0), ("bf16", 64, 0), ("bf16", 128, 32), ("fp32", 128, 0), ("fp32", 64, 32)]


@pytest.mark.parametrize("dtype,d,chunk", KINDS)
@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (1, 2, 2), (2, 9, 31), (1, 9, 127), (1, 9, 128), (2, 3, 129), (1, 9, 400),
                                   (1, 2, 1500)])
@pytest.mark.parametrize("kind", ["ladder", "mix"])
def test_prefill(la, B, H, N, dtype, d, chunk, kind):
    q, k, v = synth.dense(B, H, N, d, dtype, seed=N + d)
    g = ladder(H, kind)
    s0 = states(B, H, d, N) if (N + H) % 2 else None
    o, s = run_prefill(la, q, k, v, g, s0, chunk=chunk)
    ro, rs = od.recurrent(q, k, v, g, s0)
    assert_out(o, ro, q.dtype, 2)
    assert_state(s, rs, 2, tol=STATE)


@pytest.mark.parametrize("dtype,d,B,H,N", [("bf16", 128, 2, 80, 260), ("bf16", 64, 3, 110, 300), ("fp32", 64, 1, 170, 70)])
def test_prefill_more_units_than_sms(la, dtype, d, B, H, N):
    q, k, v = synth.dense(B, H, N, d, dtype, seed=5)
    g, s0 = ladder(H), states(B, H, d, 6)
    o, s = run_prefill(la, q, k, v, g, s0)
    ro, rs = od.recurrent(q, k, v, g, s0)
    assert_out(o, ro, q.dtype, 2)
    assert_state(s, rs, 2, tol=STATE)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 64)])
@pytest.mark.parametrize("segments", ["1", "2", "5"])
def test_prefill_segments(la, monkeypatch, dtype, d, segments):
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", segments)
    B, H, N = 1, 9, 1100
    q, k, v = synth.dense(B, H, N, d, dtype, seed=9)
    g, s0 = ladder(H, "mix"), states(B, H, d, 10)
    o, s = run_prefill(la, q, k, v, g, s0)
    ro, rs = od.recurrent(q, k, v, g, s0)
    assert_out(o, ro, q.dtype, 2)
    assert_state(s, rs, 2, tol=STATE)


def test_no_decay_equals_the_call_without(la):
    """g = 0 weighs every token with 1: the same sums as without a decay (each side is within the bars of the exact
    result, so they are within twice those of each other)."""
    q, k, v = synth.dense(1, 2, 700, 128, "bf16", seed=3)
    o, s = run_prefill(la, q, k, v, torch.zeros(2), None)
    o1, s1 = la.prefill(*cuda(q, k, v))
    assert rel_per_unit(o, o1, 2).max() <= 1e-2
    assert rel_per_unit(s, s1, 2).max() <= 2 * STATE


def test_prefill_of_no_tokens(la):
    q = torch.zeros(1, 2, 0, 128, dtype=torch.bfloat16, device="cuda")
    s0 = torch.randn(1, 2, 128, 128, device="cuda")
    g = torch.tensor([-0.5, -math.inf], device="cuda")
    o, s = la.prefill(q, q, q, s0, log_decay=g)
    assert o.shape == q.shape and torch.equal(s, s0)
    dq, dk, dv, ds0 = la.prefill_backward(q, q, q, q, None, s0, log_decay=g)
    assert torch.equal(ds0, s0)


def test_slow_decay_over_many_chunks(la):
    """exp(128 g) repeats at every chunk: an error of one rounding in it would show here (256 chunks)."""
    d, N = 64, 32768
    q, k, v = synth.dense(1, 2, N, d, "bf16", seed=21)
    g = torch.tensor([-1e-5, -3e-4])
    s0 = states(1, 2, d, 22) * 50
    for dtype in (torch.bfloat16, torch.float32):
        o, s = run_prefill(la, *(x.to(dtype) for x in (q, k, v)), g, s0)
        ro, rs = od.recurrent(q, k, v, g, s0)
        assert_out(o, ro, dtype, 2)
        # sqrt(32768) 2^-24 = 1.1e-5
        assert_state(s, rs, 2, tol=1.1e-5)


def _packed(lens, H, d, dtype, seed, slack=0, pool_n=3):
    cu = synth.cu_seqlens(lens)
    T = int(cu[-1]) + slack
    q, k, v = synth.qkv((T, H, d), d, dtype, seed=seed)
    pool = states(pool_n, H, d, seed + 1)
    idx = torch.tensor([(i % (pool_n + 1)) - 1 for i in range(len(lens))], dtype=torch.int32)
    return cu, q, k, v, pool, idx


@pytest.mark.parametrize("dtype,d,chunk", KINDS)
@pytest.mark.parametrize("lens", [[1], [0], [130, 0, 7, 128, 1, 300], [5] * 40, [1200, 3]])
def test_varlen(la, dtype, d, chunk, lens):
    """Rows behind the last sequence hold NaN in every input and stay as they were in the output."""
    H, slack = 9, 37
    cu, q, k, v, pool, idx = _packed(lens, H, d, dtype, seed=len(lens) + d, slack=slack)
    used = int(cu[-1])
    for t in (q, k, v):
        t[used:] = float("nan")
    g = ladder(H, "mix")
    o = torch.full(v.shape, 7.0, dtype=q.dtype, device="cuda")
    _, s = la.prefill_varlen(*cuda(q, k, v, cu, pool, idx), out=o, log_decay=g.cuda(), chunk=chunk)
    torch.cuda.synchronize()
    assert la.device_status() == 0
    assert (o[used:] == 7.0).all()
    ro, rs = od.varlen(q, k, v, cu, g, pool, idx)
    assert_varlen_out(o[:used].cpu(), ro[:used], cu, q.dtype)
    assert_state(s.cpu(), rs, 2, tol=STATE)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 128)])
@pytest.mark.parametrize("segments", ["1", "3"])
def test_varlen_segments(la, monkeypatch, dtype, d, segments):
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", segments)
    H = 3
    cu, q, k, v, pool, idx = _packed([1000, 1, 0, 517, 128], H, d, dtype, seed=31)
    g = ladder(H, "mix")
    o, s = la.prefill_varlen(*cuda(q, k, v, cu, pool, idx), log_decay=g.cuda())
    torch.cuda.synchronize()
    ro, rs = od.varlen(q, k, v, cu, g, pool, idx)
    assert_varlen_out(o.cpu(), ro, cu, q.dtype)
    assert_state(s.cpu(), rs, 2, tol=STATE)


@pytest.mark.parametrize("dtype,state", [("bf16", "float32"), ("fp32", "float32"), ("bf16", "bfloat16"), ("bf16", "float16"),
                                         ("bf16", "float8_e4m3fn"), ("bf16", "float8_e5m2")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 9)])
def test_decode(la, dtype, state, d, B, H):
    """Every stored element is one rounding (half a step of its format; the smallest formats' subnormals have a fixed
    step) of a value with two fp32 roundings before it; o reads the stored state."""
    sdt = getattr(torch, state)
    q, k, v = synth.qkv((B, H, d), d, dtype, seed=d + H)
    g = ladder(H, "mix")
    S = states(B, H, d, 3).to(sdt).cuda()
    for step in range(3):
        before = S.float().cpu()
        o = la.decode_step(*cuda(q, k, v), S, log_decay=g.cuda())
        torch.cuda.synchronize()
        got = S.float().cpu()
        _, rs = od.decode(q, k, v, before, g)
        fi = torch.finfo(sdt)
        parts = np.abs(od.decode(q * 0, k * 0, v, before, g)[1]) + np.abs(od.decode(q, k, v, before * 0, g)[1])
        tol = 4 * 2.0 ** -24 * parts
        if state != "float32":
            tol = tol * 1.01 + np.maximum(np.abs(rs) * fi.eps / 2, float(fi.smallest_normal) * fi.eps / 2) * 1.0001
        assert (np.abs(to64(got) - rs) <= tol).all(), f"step {step}"
        ro = np.matmul(to64(q)[..., None, :], to64(got))[..., 0, :]
        if dtype == "bf16":
            assert_out(o.cpu(), ro, q.dtype, 2)
        else:
            # a sum of d products in any order: d roundings of partial sums, each at most 2^-24 of the sum of the
            # products' magnitudes (not of o, which cancels: with full decay o = (q . k) v)
            size = np.matmul(np.abs(to64(q))[..., None, :], np.abs(to64(got)))[..., 0, :]
            assert (np.abs(to64(o.cpu()) - ro) <= d * 2.0 ** -24 * size).all()


def _check_grads(got, ref, dtype):
    for x, r, n in zip(got[:3], ref[:3], ("dq", "dk", "dv")):
        assert_out(x.cpu(), r, dtype, 2, what=n)
    assert_state(got[3].cpu(), ref[3], 2, tol=STATE)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (1, 9, 33), (2, 9, 128), (1, 9, 385), (2, 2, 1100)])
def test_backward(la, dtype, d, B, H, N):
    q, k, v = synth.dense(B, H, N, d, dtype, seed=N)
    dout = synth.dense(B, H, N, d, dtype, seed=N + 1)[2]
    g = ladder(H, "mix")
    s0, ds = (states(B, H, d, 4), states(B, H, d, 5)) if N % 2 else (None, None)
    got = la.prefill_backward(*cuda(q, k, v, dout, s0, ds), log_decay=g.cuda())
    torch.cuda.synchronize()
    assert la.device_status() == 0
    _check_grads(got, od.backward(q, k, v, dout, g, s0, ds), q.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("segments", ["1", "2", "4"])
def test_backward_segments(la, monkeypatch, dtype, segments):
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", segments)
    B, H, N, d = 1, 9, 900, 64
    q, k, v = synth.dense(B, H, N, d, dtype, seed=41)
    dout = synth.dense(B, H, N, d, dtype, seed=42)[2]
    g, s0, ds = ladder(H, "mix"), states(B, H, d, 43), states(B, H, d, 44)
    got = la.prefill_backward(*cuda(q, k, v, dout, s0, ds), log_decay=g.cuda())
    torch.cuda.synchronize()
    _check_grads(got, od.backward(q, k, v, dout, g, s0, ds), q.dtype)


def test_backward_against_differences(la):
    """Central differences of a loss through the fp32 prefill: the loss is linear in each single input, so the quotient
    is exact up to fp32 rounding of the loss's terms."""
    B, H, N, d = 1, 2, 70, 64
    q, k, v = synth.dense(B, H, N, d, "fp32", seed=51)
    dout = synth.dense(B, H, N, d, "fp32", seed=52)[2]
    g, s0, ds = torch.tensor([-0.05, -0.7]), states(B, H, d, 53), states(B, H, d, 54) * 0.1
    args = cuda(q, k, v, s0)
    grads = la.prefill_backward(*args[:3], dout.cuda(), args[3], ds.cuda(), log_decay=g.cuda())

    def loss(x):
        o, s = la.prefill(*x, log_decay=g.cuda())
        return float((o.double() * dout.cuda().double()).sum() + (s.double() * ds.cuda().double()).sum())

    r = np.random.default_rng(55)
    for x, grad in zip(range(4), (*grads[:3], grads[3])):
        for _ in range(4):
            direction = torch.from_numpy(r.standard_normal(args[x].shape)).float().cuda()
            up, down = ([a + (sgn * direction if i == x else 0) for i, a in enumerate(args)] for sgn in (1, -1))
            num = (loss(up) - loss(down)) / 2
            want = float((grad.double() * direction.double()).sum())
            # each loss sums 2 N d H terms of fp32 outputs, 1e-4 off in the 2-norm at most (parity.FP32_O_REL)
            scale = math.sqrt(2) * sum(float((la.prefill(*a, log_decay=g.cuda())[0].double() * dout.cuda()).norm())
                                       for a in (up, down))
            assert abs(num - want) <= 1e-4 * scale + 1e-6 * abs(want)


def test_prefill_then_decode_equals_one_prefill(la):
    """A prompt, then its last tokens one at a time, is the prompt with them: state and outputs."""
    B, H, N, d, steps = 1, 3, 300, 128, 5
    q, k, v = synth.dense(B, H, N + steps, d, "fp32", seed=61)
    g = ladder(H)
    o_all, s_all = la.prefill(*cuda(q, k, v), log_decay=g.cuda())
    o, s = la.prefill(*(x[:, :, :N].contiguous().cuda() for x in (q, k, v)), log_decay=g.cuda())
    for t in range(N, N + steps):
        ot = la.decode_step(*(x[:, :, t].contiguous().cuda() for x in (q, k, v)), s, log_decay=g.cuda())
        assert rel_per_unit(ot.cpu(), o_all[:, :, t].cpu(), 2).max() <= 2e-4  # both within 1e-4 of the exact outputs
    assert rel_per_unit(s.cpu(), s_all.cpu(), 2).max() <= 2 * STATE


def test_two_streams_and_repeat(la):
    """Calls on two streams with workspaces of their own, and repeated calls, agree bit for bit with a lone call."""
    q, k, v = cuda(*synth.dense(1, 4, 3000, 128, "bf16", seed=71))
    g = ladder(4).cuda()
    o, s = la.prefill(q, k, v, log_decay=g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(la.prefill(q, k, v, log_decay=g))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, o) and torch.equal(b, s)


def test_captured_and_replayed(la):
    """Prefill, backward and decode in one CUDA graph, replayed on new inputs."""
    B, H, N, d = 1, 2, 2500, 64
    g = ladder(H).cuda()
    x = cuda(*synth.dense(B, H, N, d, "bf16", seed=81))
    tok = [t[:, :, 0].contiguous() for t in x]
    S = torch.zeros(B, H, d, d, device="cuda")

    def step():
        o, s = la.prefill(*x, log_decay=g)
        grads = la.prefill_backward(*x, o, None, s, log_decay=g)
        S.copy_(s)
        return o, s, *grads, la.decode_step(*tok, S, log_decay=g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (82, 83):
        for a, b in zip(x, synth.dense(B, H, N, d, "bf16", seed=seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [S.clone()]
        want = list(step()) + [S]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_validate_finds_bad_decays(la, monkeypatch):
    monkeypatch.setenv("LA_VALIDATE", "1")
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (1e-3, float("nan"), math.inf):
        with pytest.raises(la.LAError):
            la.prefill(x, x, x, log_decay=torch.tensor([-1.0, bad], device="cuda"))
    la.prefill(x, x, x, log_decay=torch.tensor([0.0, -math.inf], device="cuda"))


def test_wrapper_refusals(la):
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(2, device="cuda")
    for bad in (g[:1], g.double(), torch.zeros(2, 1, device="cuda")):
        with pytest.raises((ValueError, TypeError)):
            la.prefill(x, x, x, log_decay=bad)
    with pytest.raises(ValueError):
        la.prefill(x, x, x, log_decay=g.cpu())
    with pytest.raises(ValueError):
        la.prefill(x, x, x, log_decay=g, phi="relu")
    with pytest.raises(ValueError):
        la.prefill(x, x, x, log_decay=g, out=torch.empty(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda"))


# sizes whose (unit, 64 value columns) items leave SMs idle in the last turn: a
# unit's chunks are then divided between two CTAs, which hand its state on
SHARED = [(128, 1, 76, 700), (128, 5, 15, 1025), (128, 3, 50, 640), (64, 1, 149, 900), (64, 10, 20, 1300)]


@pytest.mark.parametrize("d,B,H,N", SHARED)
@pytest.mark.parametrize("resume", [False, True])
def test_prefill_shared_out_by_chunks(la, d, B, H, N, resume):
    q, k, v = synth.dense(B, H, N, d, "bf16", seed=23)
    g = ladder(H, "mix")
    s0 = states(B, H, d, 24) if resume else None
    assert la.lib.la_prefill_decay_workspace_size(B, H, N, d, d, la._abi.LA_BF16) > 0
    o, s = run_prefill(la, q, k, v, g, s0)
    # without the workspace whole items run in turn: the same arithmetic
    c = cuda(q, k, v, s0, g)
    o1, s1 = torch.empty_like(c[0]), torch.empty(B, H, d, d, device="cuda")
    ptr = [None if t is None else t.data_ptr() for t in c]
    st = torch.cuda.current_stream().cuda_stream
    assert la.lib.la_prefill_decay(ptr[0], ptr[1], ptr[2], o1.data_ptr(), ptr[3], s1.data_ptr(), ptr[4], B, H, N, d, d,
                                   la._abi.LA_BF16, 0, None, 0, st) == 0
    torch.cuda.synchronize()
    assert torch.equal(o, o1.cpu()) and torch.equal(s, s1.cpu())
    ro, rs = od.recurrent(q, k, v, g, s0)
    assert_out(o, ro, q.dtype, 2)
    assert_state(s, rs, 2, tol=STATE)


@pytest.mark.parametrize("d,B,H,N", SHARED[1:4])
def test_backward_shared_out_by_chunks(la, d, B, H, N):
    q, k, v = synth.dense(B, H, N, d, "bf16", seed=25)
    do = synth.dense(B, H, N, d, "bf16", seed=26)[2]
    g, s0, ds = ladder(H, "mix"), states(B, H, d, 27), states(B, H, d, 28)
    c = cuda(q, k, v, do, s0, ds, g)
    got = la.prefill_backward(*c[:6], log_decay=c[6])
    want = [torch.empty_like(t) for t in got]
    assert la.lib.la_prefill_decay_backward(*(t.data_ptr() for t in c), *(t.data_ptr() for t in want), B, H, N, d, d,
                                            la._abi.LA_BF16, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert la.device_status() == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_shared_out_captured_and_on_two_streams(la):
    B, H, N, d = 3, 50, 640, 128
    q, k, v = (t.cuda() for t in synth.dense(B, H, N, d, "bf16", seed=29))
    g = ladder(H).cuda()
    want = la.prefill(q, k, v, log_decay=g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        la.prefill(q, k, v, log_decay=g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = la.prefill(q, k, v, log_decay=g)
    for _ in range(3):
        o.zero_()
        s.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            o2, s2 = la.prefill(q, k, v, log_decay=g)
        torch.cuda.synchronize()
        for a, b in zip(want, (o, s)):
            assert torch.equal(a, b)
        for a, b in zip(want, (o2, s2)):
            assert torch.equal(a, b)
    assert la.device_status() == 0


@pytest.mark.parametrize("d,B,H,N", [(64, 1, 3, 777), (128, 2, 9, 200)])
def test_fp32_backward_without_a_workspace(la, d, B, H, N):
    q, k, v = synth.dense(B, H, N, d, "fp32", seed=61)
    dout = synth.dense(B, H, N, d, "fp32", seed=62)[2]
    g, s0, ds = ladder(H, "mix"), states(B, H, d, 63), states(B, H, d, 64)
    c = cuda(q, k, v, dout, s0, ds, g)
    got = [torch.empty_like(t) for t in (*c[:3], c[4])]
    assert la.lib.la_prefill_decay_backward(*(t.data_ptr() for t in c), *(t.data_ptr() for t in got), B, H, N, d, d,
                                            la._abi.LA_FP32, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    _check_grads(got, od.backward(q, k, v, dout, g, s0, ds), q.dtype)
