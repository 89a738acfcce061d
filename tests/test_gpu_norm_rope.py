"""The norm of query and key heads with rotation, and its gradients, against
the fp64 oracle.

Tolerance of one fp32 output: the sum of squares (log2(d) + 1 = 8 roundings),
the reciprocal root (2 ulp), two products, the cosine and sine (1 ulp each and
the angle's rounding, 2^-25 turns), three roundings of the rotation: together
below 2^-20 of the pair's size; E takes 2^-19 of the row's largest value times
2.  bf16 adds half a step of the result, 2^-8.  Weight gradients are fp32 sums
of n terms: sqrt(n) 2^-24 of the sum of magnitudes is far above what is seen;
2^-18 of it is allowed.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import norm_rope as onr
from tests.parity import to64

pytestmark = pytest.mark.gpu
E = 2.0 ** -19


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


def freqs(rot):
    half = rot // 2
    return None if rot == 0 else (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float()


def inputs(B, N, Hq, Hk, d, dtype, seed, wdt=None):
    g = torch.Generator().manual_seed(seed)
    dt = synth.torch_dtype(dtype)
    q, k = (torch.randn(B, H, N, d, generator=g).to(dt) for H in (Hq, Hk))
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)).to(wdt or dt) for _ in range(2))
    dyq, dyk = (torch.randn(B, H, N, d, generator=g).to(dt) for H in (Hq, Hk))
    return q, k, wq, wk, dyq, dyk


def close(got, ref, dtype, scale=1.0):
    got = to64(got)
    tol = 2 * E * scale * np.maximum(np.abs(ref).max(-1, keepdims=True), 1e-30)
    if dtype == "bf16":
        tol = tol + np.abs(ref) * 2.0 ** -8
    assert got.shape == ref.shape and np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(np.abs(got - ref) / tol):.2f} of the bound"


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check(la, q, k, wq, wk, dyq, dyk, rot, pos, dtype, interleaved, eps=1e-6, shape=lambda t: t.cuda()):
    """pos: numpy int64 [N] or [B, N]"""
    f = freqs(rot)
    R = onr.rotation(q.shape[-1], f, pos, interleaved)
    R = R if pos.ndim == 1 else R[:, None]
    a = [shape(q), shape(k), *cuda(wq, wk, f, torch.from_numpy(pos))]
    yq, yk = la.qk_norm_rope(*a, eps=eps, interleaved=interleaved)
    dq, dk, dwq, dwk = la.qk_norm_rope_backward(shape(dyq), shape(dyk), *a, eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    for x, w, y, dy, dx, dw in ((q, wq, yq, dyq, dq, dwq), (k, wk, yk, dyk, dk, dwk)):
        assert y.is_contiguous() and y.shape == x.shape
        close(y.cpu(), onr.forward(x, w, R, eps), dtype)
        rdx, rdw = onr.backward(dy, x, w, R, eps)
        # dx is a difference of terms of size r |w g|
        r = 1 / np.sqrt((to64(x) ** 2).mean(-1, keepdims=True) + eps)
        big = (r * np.abs(to64(w)).max() * np.abs(to64(dy)).max(-1, keepdims=True) * 2)
        tol = 4 * E * big + (np.abs(rdx) * 2.0 ** -8 if dtype == "bf16" else 0)
        assert (np.abs(to64(dx.cpu()) - rdx) <= tol).all()
        xh = to64(x) * r
        terms = np.abs(to64(dy)).max(-1, keepdims=True) * 2 * np.abs(xh)
        assert (np.abs(to64(dw.cpu()) - rdw) <= 2.0 ** -18 * terms.reshape(-1, x.shape[-1]).sum(0) + 1e-30).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("rot", [0, 16, 48, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_rotated_dims(la, dtype, d, rot, interleaved):
    if rot > d:
        pytest.skip("rot > d")
    x = inputs(2, 19, 5, 3, d, dtype, seed=rot + d)
    check(la, *x, rot, np.arange(100, 119), dtype, interleaved)


@pytest.mark.parametrize("B,N,Hq,Hk", [(1, 1, 1, 1), (1, 1, 1, 0), (1, 3, 0, 2), (3, 1, 64, 64), (1, 200, 1, 1), (2, 65, 7, 1),
                                       (1, 33, 130, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sizes(la, B, N, Hq, Hk, dtype):
    x = inputs(B, N, Hq, Hk, 128, dtype, seed=N)
    check(la, *x, 128, np.arange(N), dtype, False)


@pytest.mark.parametrize("dtype,Hq,Hk", [("bf16", 1, 2), ("bf16", 3, 1), ("fp32", 2, 1)])
def test_many_tokens_of_few_heads(la, dtype, Hq, Hk):
    # (enough rows for several of them per thread)
    x = inputs(4, 5003, Hq, Hk, 64, dtype, seed=7)
    check(la, *x, 32, np.arange(5003), dtype, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_far_positions_of_each_sequence(la, dtype):
    """Angles of 10^9 radians: the frequencies are fp32 values, their products with the position are exact in double."""
    x = inputs(3, 6, 2, 2, 128, dtype, seed=1)
    pos = np.array([[0], [1 << 20], [(1 << 31) - 10]], dtype=np.int64) + np.arange(6)
    check(la, *x, 128, pos, dtype, False)
    check(la, *x, 128, -pos, dtype, True)


def test_positions_of_32_bits_strided_or_left_out(la):
    q, k, wq, wk, _, _ = cuda(*inputs(2, 9, 2, 2, 64, "fp32", seed=2))
    f = freqs(64).cuda()
    want = la.qk_norm_rope(q, k, wq, wk, f, torch.arange(9, device="cuda"))
    for pos in (None, torch.arange(9, device="cuda", dtype=torch.int32), torch.arange(9, device="cuda").expand(2, 9),
                torch.arange(18, device="cuda").view(9, 2)[:, 0].div(2, rounding_mode="floor")):
        got = la.qk_norm_rope(q, k, wq, wk, f, pos)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layouts(la):
    """Slices of one projection's output, packed tokens and decode tokens give what contiguous heads give; gradients
    are written into slices too."""
    B, N, Hq, Hk, d = 2, 21, 4, 2, 128
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(B, N, Hq + 2 * Hk, d, generator=g).bfloat16().cuda()
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    wq, wk = (torch.rand(d, generator=g).bfloat16().cuda() for _ in range(2))
    f, pos = freqs(64).cuda(), torch.randint(0, 1000, (B, N), generator=g).cuda()
    want = la.qk_norm_rope(q.contiguous(), k.contiguous(), wq, wk, f, pos)
    got = la.qk_norm_rope(q, k, wq, wk, f, pos)
    assert all(torch.equal(a, b) and a.is_contiguous() for a, b in zip(got, want))
    tok = qkv.view(B * N, Hq + 2 * Hk, d)
    packed = la.qk_norm_rope(tok[:, :Hq], tok[:, Hq:Hq + Hk], wq, wk, f, pos.view(-1))
    for a, b in zip(packed, want):
        assert torch.equal(a.view(B, N, -1, d).transpose(1, 2), b)
    dy = [torch.randn(t.shape, generator=g).bfloat16().cuda() for t in want]
    ref = la.qk_norm_rope_backward(*dy, q.contiguous(), k.contiguous(), wq, wk, f, pos)
    dqkv = torch.full_like(qkv, 5.0)
    out = la.qk_norm_rope_backward(*dy, q, k, wq, wk, f, pos, dq=dqkv[:, :, :Hq].transpose(1, 2),
                                   dk=dqkv[:, :, Hq:Hq + Hk].transpose(1, 2))
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert (dqkv[:, :, Hq + Hk:] == 5.0).all()


def test_weights_in_fp32(la):
    x = inputs(1, 40, 3, 3, 128, "bf16", seed=4, wdt=torch.float32)
    check(la, *x, 64, np.arange(40), "bf16", False)


def test_many_rows_and_repeats(la):
    """More rows than one pass of the backward's grid; the weight gradients are the same bits every time."""
    x = inputs(1, 3000, 16, 16, 64, "bf16", seed=5)
    check(la, *x, 32, np.arange(3000), "bf16", True)
    q, k, wq, wk, dyq, dyk = cuda(*x)
    runs = [la.qk_norm_rope_backward(dyq, dyk, q, k, wq, wk, freqs(32).cuda()) for _ in range(3)]
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


def test_no_tokens(la):
    q = torch.zeros(1, 2, 0, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    a, b = la.qk_norm_rope(q, q, w, w, freqs(128).cuda())
    assert a.shape == q.shape == b.shape
    out = la.qk_norm_rope_backward(q, q, q, q, w, w, freqs(128).cuda())
    assert (out[2] == 0).all() and (out[3] == 0).all()


def test_large_and_small_values(la):
    """Rows of zeros give zeros (eps > 0); values of 1e15 and 1e-15 keep their norm."""
    x = inputs(1, 4, 1, 1, 128, "fp32", seed=6)
    for scale in (0.0, 1e-15, 1e15):
        q, k = x[0] * scale, x[1] * scale
        f = freqs(128)
        yq, _ = la.qk_norm_rope(*cuda(q, k, x[2], x[3], f), eps=1e-30)
        close(yq.cpu(), onr.forward(q, x[2], onr.rotation(128, f, np.arange(4)), 1e-30), "fp32")


def test_captured_and_replayed(la):
    x = cuda(*inputs(1, 50, 4, 4, 128, "bf16", seed=7))
    f = freqs(128).cuda()
    pos = torch.arange(50, device="cuda")

    def step():
        y = la.qk_norm_rope(*x[:4], f, pos)
        return (*y, *la.qk_norm_rope_backward(x[4], x[5], *x[:4], f, pos))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    pos += 77
    for a, b in zip(x, inputs(1, 50, 4, 4, 128, "bf16", seed=8)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_refusals(la):
    q = torch.zeros(1, 2, 4, 128, device="cuda")
    w, f = torch.ones(128, device="cuda"), freqs(128).cuda()
    bad = [
        lambda: la.qk_norm_rope(q, q[:, :, :3], w, w, f),
        lambda: la.qk_norm_rope(q, q, w[:64], w, f),
        lambda: la.qk_norm_rope(q, q, w.bfloat16(), w, f),
        lambda: la.qk_norm_rope(q, q, w.half(), w.half(), f),
        lambda: la.qk_norm_rope(q, q, w, w, f.double()),
        lambda: la.qk_norm_rope(q, q, w, w, f[:60]),                                 # rot not a multiple of 16
        lambda: la.qk_norm_rope(q, q, w, w, f.repeat(2)),                            # rot > d
        lambda: la.qk_norm_rope(q, q, w, w, f, torch.zeros(3, device="cuda", dtype=torch.int64)),
        lambda: la.qk_norm_rope(q, q, w, w, f, torch.zeros(4, device="cuda")),
        lambda: la.qk_norm_rope(q, q, w, w, f, torch.zeros(4, dtype=torch.int64)),
        lambda: la.qk_norm_rope(q[0], q[0], w, w, f),                                # packed without positions
        lambda: la.qk_norm_rope(q.transpose(2, 3), q.transpose(2, 3), w, w, f),
        lambda: la.qk_norm_rope(q, q.bfloat16(), w, w, f),
        lambda: la.qk_norm_rope(q.double(), q.double(), w, w, f),
        lambda: la.qk_norm_rope(q[..., :96].contiguous(), q[..., :96].contiguous(), w[:96], w[:96], f[:32]),
        lambda: la.qk_norm_rope(q, q, w, w, f, eps=-1.0),
        lambda: la.qk_norm_rope(q, q, w, w, f, q_out=q[:, :1]),
        lambda: la.qk_norm_rope_backward(q[:, :1], q, q, q, w, w, f),
        # rows that do not start on 16 bytes
        lambda: la.qk_norm_rope(*[torch.zeros(1, 4, 2, 129, device="cuda")[..., :128].transpose(1, 2)] * 2, w, w, f),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, la.LAError)):
            call()
            pytest.fail(f"call {i} was not refused")
