"""The operators of a decayed linear-attention layer together, as a user runs
them: projection -> norm and rotation -> decayed attention, for prompts and then
token by token (serving), and forward with all gradients (training)."""
import numpy as np
import pytest
import torch

from oracle import decay as od
from oracle import norm_rope as onr
from tests.parity import assert_out, assert_state, rel_per_unit, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


D, ROT = 128, 64


def layer(H, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    wq, wk = (((1 + 0.2 * torch.randn(D, generator=g)) * D ** -0.5).to(dtype) for _ in range(2))
    f = (10000.0 ** (-torch.arange(ROT // 2, dtype=torch.float64) / (ROT // 2))).float()
    return g, wq, wk, f, -torch.exp2(-8.0 * torch.arange(1, H + 1) / H)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_serving(la, dtype):
    """A packed batch of prompts (one empty, one resumed) from one projection's output, then decode steps at each
    sequence's next positions, against the oracles on the layer's own queries and keys."""
    H, lens, steps = 4, [150, 0, 1, 130], 3
    g, wq, wk, f, ld = layer(H, 1, dtype)
    cu = [0, 150, 150, 151, 281]
    T, n = cu[-1], len(lens)
    first = [5, 0, 1 << 20, 64]  # position of each sequence's first token
    pos = torch.cat([p + torch.arange(x) for p, x in zip(first, lens)])
    qkv = torch.randn(T, 3 * H, D, generator=g).to(dtype)
    pool = torch.randn(1, H, D, D, generator=g) * 0.3
    idx = torch.tensor([-1, 0, -1, 0], dtype=torch.int32)
    a = qkv.cuda()
    q, k = la.qk_norm_rope(a[:, :H], a[:, H:2 * H], wq.cuda(), wk.cuda(), f.cuda(), pos.cuda())
    o, S = la.prefill_varlen(q, k, a[:, 2 * H:].contiguous(), torch.tensor(cu, dtype=torch.int32).cuda(), pool.cuda(),
                             idx.cuda(), log_decay=ld.cuda())
    outs = []
    toks = [torch.randn(n, 3 * H, D, generator=g).to(dtype) for _ in range(steps)]
    where = [torch.tensor([p + x + t for p, x in zip(first, lens)]) for t in range(steps)]
    for x, at in zip(toks, where):
        x = x.cuda()
        qt, kt = la.qk_norm_rope(x[:, :H], x[:, H:2 * H], wq.cuda(), wk.cuda(), f.cuda(), at.cuda())
        outs.append((qt, kt, la.decode_step(qt, kt, x[:, 2 * H:].contiguous(), S, log_decay=ld.cuda())))
    torch.cuda.synchronize()
    assert la.device_status() == 0
    # the norm and rotation: one rounding (bf16) or fp32 arithmetic of the oracle's values
    R = onr.rotation(D, f, pos.numpy())[:, None]
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for got, x, w in ((q, qkv[:, :H], wq), (k, qkv[:, H:2 * H], wk)):
        ref = onr.forward(x, w, R, 1e-6)
        assert (np.abs(to64(got.cpu()) - ref) <= half * np.abs(ref) + 2.0 ** -18 * np.abs(ref).max()).all()
    # the attention, on the queries and keys that it was given
    ro, rS = od.varlen(q.cpu(), k.cpu(), qkv[:, 2 * H:], cu, ld, pool, idx)
    for s in range(n):
        if lens[s]:
            part = slice(cu[s], cu[s + 1])
            assert_out(o[part].cpu().transpose(0, 1), np.swapaxes(ro[part], 0, 1), dtype, 1)
    for x, (qt, kt, ot) in zip(toks, outs):
        ro, rS = od.decode(qt.cpu(), kt.cpu(), x[:, 2 * H:], rS, ld)
        assert_out(ot.cpu(), ro, dtype, 2)
    assert_state(S.cpu(), rS, 2, tol=5e-6)


def test_training_gradients(la):
    """Gradients of the whole chain in fp32 (inputs, norm weights, values, first state) against autograd of the
    formulas in 64 bits: every operator is within 1e-4 in the 2-norm, five of them follow one another."""
    B, N, H = 2, 70, 3
    g, wq, wk, f, ld = layer(H, 2, torch.float32)
    qk = torch.randn(B, N, 2 * H, D, generator=g)
    v, do = (torch.randn(B, H, N, D, generator=g) for _ in range(2))
    s0, ds = (torch.randn(B, H, D, D, generator=g) * 0.2 for _ in range(2))
    a = qk.cuda()
    x, y = a[:, :, :H].transpose(1, 2), a[:, :, H:].transpose(1, 2)
    w = wq.cuda(), wk.cuda()
    q, k = la.qk_norm_rope(x, y, *w, f.cuda())
    la.prefill(q, k, v.cuda(), s0.cuda(), log_decay=ld.cuda())
    dq, dk, dv, ds0 = la.prefill_backward(q, k, v.cuda(), do.cuda(), s0.cuda(), ds.cuda(), log_decay=ld.cuda())
    dqk = torch.empty_like(a)
    _, _, dwq, dwk = la.qk_norm_rope_backward(dq, dk, x, y, *w, f.cuda(), dq=dqk[:, :, :H].transpose(1, 2),
                                              dk=dqk[:, :, H:].transpose(1, 2))
    torch.cuda.synchronize()
    # the same by autograd in 64 bits
    leaves = [t.double().requires_grad_(True) for t in (qk, wq, wk, v, s0)]
    rqk, rwq, rwk, rv, rs0 = leaves
    ang = torch.arange(N, dtype=torch.float64)[:, None] * f.double()
    c, s = torch.cos(ang), torch.sin(ang)

    def norm_rope(t, wt):
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * wt
        p, r, rest = t[..., :ROT // 2], t[..., ROT // 2:ROT], t[..., ROT:]
        return torch.cat((p * c - r * s, r * c + p * s, rest), -1)

    rq, rk = norm_rope(rqk[:, :, :H].transpose(1, 2), rwq), norm_rope(rqk[:, :, H:].transpose(1, 2), rwk)
    t = torch.arange(1, N + 1, dtype=torch.float64)
    gd = ld.double()[:, None]
    gap = t[:, None] - t[None, :]
    mask = torch.exp(gd[..., None] * gap.clamp(min=0)) * (gap >= 0)
    o = (rq @ rk.transpose(2, 3) * mask) @ rv + torch.exp(gd * t)[..., None] * (rq @ rs0)
    S = (rk * torch.exp(gd * (N - t))[..., None]).transpose(2, 3) @ rv + torch.exp(gd * N)[..., None] * rs0
    loss = (o * do.double()).sum() + (S * ds.double()).sum()
    ref = torch.autograd.grad(loss, leaves)
    for got, want, lead in ((dqk, ref[0], 1), (dwq, ref[1], 0), (dwk, ref[2], 0), (dv, ref[3], 2), (ds0, ref[4], 2)):
        assert rel_per_unit(got.cpu(), want.numpy(), lead).max() <= 5e-4


def test_layer_in_one_graph(la):
    """Norm, rotation and decode of one token captured once and replayed at moving positions."""
    B, H, dtype = 3, 4, torch.bfloat16
    g, wq, wk, f, ld = layer(H, 3, dtype)
    x = torch.randn(B, 3 * H, D, generator=g).to(dtype).cuda()
    pos = torch.tensor([0, 7, 1 << 20]).cuda()
    S = torch.zeros(B, H, D, D, device="cuda")
    w = wq.cuda(), wk.cuda(), f.cuda()
    ld = ld.cuda()

    def token():
        q, k = la.qk_norm_rope(x[:, :H], x[:, H:2 * H], *w, pos)
        return la.decode_step(q, k, x[:, 2 * H:].contiguous(), S, log_decay=ld)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token()
    xs = [torch.randn(B, 3 * H, D, generator=g).to(dtype).cuda() for _ in range(4)]
    S.zero_()
    pos.copy_(torch.tensor([0, 7, 1 << 20]))
    got = []
    for y in xs:
        x.copy_(y)
        graph.replay()
        got.append(out.clone())
        pos += 1
    last = S.clone()
    S.zero_()
    pos.copy_(torch.tensor([0, 7, 1 << 20]))
    for y, want in zip(xs, got):
        x.copy_(y)
        assert torch.equal(token(), want)
        pos += 1
    assert torch.equal(S, last)
