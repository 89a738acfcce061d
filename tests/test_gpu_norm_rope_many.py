"""The norm with rotation on more rows than one per thread fills the GPU with: the
instances of several rows per thread, forward and backward, and positions of any
strides.

The reference is written with complex numbers (a pair of frequency i is one
number, turned by exp(i p f)), in 64 bits, for sizes where a matrix per token would
not do; it is compared with the oracle's matrices first.  Tolerances as derived in
test_gpu_norm_rope.py.
"""
import numpy as np
import pytest
import torch

from oracle import norm_rope as onr
from tests.parity import to64
from tests.test_gpu_norm_rope import E, close, freqs, inputs

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


def turn(x, f, pos, interleaved, back=False):
    """x [B, H, N, d] turned by the positions [B, N]."""
    half = len(f)
    if half == 0:
        return x
    z = np.exp((-1j if back else 1j) * to64(pos)[:, None, :, None] * to64(f))
    y = x.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    c = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = c.real, c.imag
    return y


def reference(x, w, dy, f, pos, interleaved):
    x, w, dy = to64(x), to64(w), to64(dy)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    xh, g = x * r, turn(dy, f, pos, interleaved, back=True)
    dx = r * (w * g - xh * (w * g * xh).mean(-1, keepdims=True))
    return turn(xh * w, f, pos, interleaved), dx, (g * xh).reshape(-1, x.shape[-1]).sum(0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [32, 64])
def test_the_reference(interleaved, rot):
    q, k, wq, _, dy, _ = inputs(2, 5, 3, 1, 64, "fp32", seed=1)
    f, pos = freqs(rot), torch.arange(7, 17).view(2, 5)
    y, dx, dw = reference(q, wq, dy, f, pos, interleaved)
    R = onr.rotation(64, f, pos.numpy(), interleaved)[:, None]
    np.testing.assert_allclose(y, onr.forward(q, wq, R, EPS), rtol=1e-12, atol=1e-14)
    rdx, rdw = onr.backward(dy, q, wq, R, EPS)
    np.testing.assert_allclose(dx, rdx, rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(dw, rdw, rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 48, 64, 128])
@pytest.mark.parametrize("Hq,Hk", [(3, 2), (2, 5)])
def test_several_rows_per_thread(la, dtype, d, interleaved, rot, Hq, Hk):
    """Entries of 1733 tokens: no entry, nor all of them, are a multiple of a block's rows, and blocks reach from one
    entry into the next."""
    if rot > d:
        pytest.skip("rot > d")
    B, N = 3, 1733
    rows = torch.cuda.get_device_properties(0).multi_processor_count * (128 // (d // (8 if dtype == "bf16" else 4) // 2)) * 4
    assert B * N * (Hq + Hk) > rows and (B * N * Hq) % 8 and N * Hq % 8
    q, k, wq, wk, dyq, dyk = inputs(B, N, Hq, Hk, d, dtype, seed=rot + d)
    f = freqs(rot)
    pos = torch.arange(N) + torch.tensor([[0], [5000], [1 << 20]])
    c = [t if t is None else t.cuda() for t in (q, k, wq, wk, f, pos)]
    # slices of one projection's output, gradients written into slices
    x = torch.cat((q, k), 1).transpose(1, 2).contiguous().cuda()
    dx = torch.full_like(x, 3.0)
    views = [(t[:, :, :Hq].transpose(1, 2), t[:, :, Hq:].transpose(1, 2)) for t in (x, dx)]
    yq, yk = la.qk_norm_rope(*views[0], *c[2:], eps=EPS, interleaved=interleaved)
    _, _, dwq, dwk = la.qk_norm_rope_backward(dyq.cuda(), dyk.cuda(), *views[0], *c[2:], eps=EPS, interleaved=interleaved,
                                              dq=views[1][0], dk=views[1][1])
    torch.cuda.synchronize()
    for x, w, dy, y, dx, dw in ((q, wq, dyq, yq, views[1][0], dwq), (k, wk, dyk, yk, views[1][1], dwk)):
        ry, rdx, rdw = reference(x, w, dy, f if f is not None else (), pos, interleaved)
        close(y.cpu(), ry, dtype)
        r = 1 / np.sqrt((to64(x) ** 2).mean(-1, keepdims=True) + EPS)
        big = r * np.abs(to64(w)).max() * np.abs(to64(dy)).max(-1, keepdims=True) * 2
        tol = 4 * E * big + (np.abs(rdx) * 2.0 ** -8 if dtype == "bf16" else 0)
        assert (np.abs(to64(dx.cpu()) - rdx) <= tol).all()
        terms = np.abs(to64(dy)).max(-1, keepdims=True) * 2 * np.abs(to64(x) * r)
        assert (np.abs(to64(dw.cpu()) - rdw) <= 2.0 ** -18 * terms.reshape(-1, d).sum(0) + 1e-30).all()


@pytest.mark.parametrize("width", [torch.int32, torch.int64])
def test_positions_of_any_strides(la, width):
    """Every second value of a longer array, columns of [N, B], one position for all tokens of an entry and one row for all
    entries."""
    B, N = 3, 37
    q, k, wq, wk, dyq, dyk = (t.cuda() for t in inputs(B, N, 2, 3, 64, "bf16", seed=2))
    f = freqs(64).cuda()
    base = (torch.arange(N) * 3 + torch.tensor([[0], [700], [90000]])).to(width).cuda()
    every = torch.stack((base, base + 17), -1)[..., 0]
    columns = torch.stack((base.t(), base.t() + 17), -1)[..., 0].t()
    alike = torch.tensor([[4], [11], [90]], dtype=width, device="cuda").expand(B, N)
    row = torch.stack((base[1], base[1] + 9), 1)[:, 0]
    assert every.stride() == (2 * N, 2) and columns.stride() == (2, 2 * B) and alike.stride() == (1, 0) and row.stride() == (2,)
    for pos in (every, columns, alike, row, row.expand(B, N)):
        plain = (pos if pos.dim() == 2 else pos.expand(B, N)).clone(memory_format=torch.contiguous_format)
        for call in (lambda p: la.qk_norm_rope(q, k, wq, wk, f, p),
                     lambda p: la.qk_norm_rope_backward(dyq, dyk, q, k, wq, wk, f, p)):
            assert all(torch.equal(a, b) for a, b in zip(call(pos), call(plain)))
        want = reference(q.cpu(), wq.cpu(), dyq.cpu(), f.cpu(), plain.cpu(), False)[0]
        close(la.qk_norm_rope(q, k, wq, wk, f, pos)[0].cpu(), want, "bf16")
    # packed tokens
    tok = q[0].transpose(0, 1).contiguous()
    got = la.qk_norm_rope(tok, tok, wq, wk, f, row)
    want = la.qk_norm_rope(tok, tok, wq, wk, f, row.contiguous())
    assert row.contiguous().stride() == (1,) and all(torch.equal(a, b) for a, b in zip(got, want))
