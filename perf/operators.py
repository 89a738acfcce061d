"""Cases of the decayed linear attention and of the query/key norm with rotation, for timing and comparison.

Two families of operators of ``long_context_linear_b200``:

* linear attention with a decay for each head, S_t = exp(g_h) S_{t-1} + k_t v_t^T, o_t = q_t S_t: ``prefill``,
  ``prefill_varlen``, ``decode_step`` and ``prefill_backward`` called with ``log_decay`` = g;
* ``qk_norm_rope`` and ``qk_norm_rope_backward``: the root-mean-square norm of every query and key head, its weight and the
  rotation by the token's position, written in the layout that the attention reads.

``own`` chooses between the framework's calls and their plain form: elementary torch operations in 32 bits (angles of the
rotation in 64), rounded once at the end.  ``exact`` holds the definitions in 64 bits, written apart from the plain form.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_CHUNK = 128  # tokens per block of the plain form


def listed():
    return [
        # one short prompt of a small fp32 layer: a latency-bound call
        {"name": "prefill_fp32_small", "op": "prefill", "B": 1, "H": 2, "N": 256, "d": 64, "dtype": "fp32", "resume": True},
        # a batch of 8K prompts, heads enough to fill the GPU
        {"name": "prefill_bf16_8k", "op": "prefill", "B": 4, "H": 32, "N": 8192, "d": 128, "dtype": "bf16", "resume": False},
        # one very long prompt: the largest call
        {"name": "prefill_bf16_128k", "op": "prefill", "B": 1, "H": 64, "N": 131072, "d": 128, "dtype": "bf16", "resume": True},
        # few narrow heads over an odd length, resumed from a cached prefix
        {"name": "prefill_bf16_odd", "op": "prefill", "B": 1, "H": 6, "N": 20011, "d": 64, "dtype": "bf16", "resume": True},
        # a packed batch of prompts of 0 to 4K tokens, some resumed from a pool of prefix states
        {"name": "varlen_bf16", "op": "varlen", "n_seq": 32, "max_len": 4096, "mix": 5, "H": 16, "d": 128,
         "dtype": "bf16"},
        # one token for each of 256 sequences: the serving step, bound by the states' bytes
        {"name": "decode_bf16", "op": "decode", "B": 256, "H": 64, "d": 128, "dtype": "bf16", "state": "fp32"},
        # a small serving batch with states stored in 16 bits: latency
        {"name": "decode_small", "op": "decode", "B": 3, "H": 16, "d": 128, "dtype": "bf16", "state": "bf16"},
        # a training step's gradients
        {"name": "backward_bf16", "op": "backward", "B": 2, "H": 32, "N": 4096, "d": 128, "dtype": "bf16"},
        # the same in fp32, narrow heads and an odd length
        {"name": "backward_fp32_odd", "op": "backward", "B": 1, "H": 3, "N": 777, "d": 64, "dtype": "fp32"},
        # queries and keys of a batch of 8K prompts, from the projections' layout to the attention's
        {"name": "norm_rope_8k", "op": "norm_rope", "B": 4, "N": 8192, "Hq": 32, "Hk": 32, "d": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "far": 0},
        # one token for each of 64 sequences at far positions: latency
        {"name": "norm_rope_decode", "op": "norm_rope", "B": 64, "N": 1, "Hq": 64, "Hk": 64, "d": 128, "rot": 64,
         "dtype": "bf16", "interleaved": False, "far": 1 << 20},
        # a training step's gradients, half of each head rotated, pairs side by side
        {"name": "norm_rope_backward", "op": "norm_rope_backward", "B": 2, "N": 4096, "Hq": 32, "Hk": 32, "d": 128,
         "rot": 64, "dtype": "bf16", "interleaved": True, "far": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "varlen", "decode", "backward", "norm_rope", "norm_rope_backward"))
    d = rng.choice((64, 128))
    # attention in fp32 computes on the CUDA cores; its calls stay shorter
    dt = rng.choice(("bf16", "bf16", "fp32"))
    small = dt == "fp32"
    if op in ("prefill", "backward"):
        B, H = rng.randint(1, 4), _log_int(rng, 1, 64)
        most = min(131072, (1 << 17 if small else 1 << 20) // (B * H))
        c = {"op": op, "B": B, "H": H, "N": _log_int(rng, 1, max(2, most)), "d": d, "dtype": dt}
        if op == "prefill":
            c["resume"] = rng.random() < 0.5
        return c
    if op == "varlen":
        return {"op": op, "n_seq": _log_int(rng, 1, 40), "max_len": _log_int(rng, 1, 1024 if small else 4096),
                "mix": rng.randrange(1000), "H": _log_int(rng, 1, 16), "d": d, "dtype": dt}
    if op == "decode":
        return {"op": op, "B": _log_int(rng, 1, 256), "H": _log_int(rng, 1, 64), "d": d, "dtype": dt,
                "state": "fp32" if small else rng.choice(("fp32", "bf16"))}
    B = _log_int(rng, 1, 64)
    Hq = _log_int(rng, 1, 64)
    return {"op": op, "B": B, "N": _log_int(rng, 1, max(1, min(8192, 32768 // B))), "Hq": Hq,
            "Hk": rng.choice((Hq, max(1, Hq // 4))), "d": d, "rot": rng.choice((16, d // 2, d)), "dtype": dt,
            "interleaved": rng.random() < 0.5, "far": rng.choice((0, 1 << 20))}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _log_decay(H, seed):
    """A geometric ladder of slopes over the heads (2^(-8 (h+1) / H)), scaled for one layer of a stack."""
    layer = 0.25 + 0.75 * random.Random(int(seed)).random()
    slopes = torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H) * layer
    return (-slopes).float().cuda()


def _state(g, shape):
    # a state that has absorbed some tens of tokens
    return _randn(g, shape, scale=0.5)


def _lengths(case):
    r = random.Random(case["mix"])
    lens = [int(round(case["max_len"] ** r.random())) for _ in range(case["n_seq"])]
    lens[r.randrange(case["n_seq"])] = case["max_len"]
    if case["n_seq"] > 3:
        lens[r.randrange(case["n_seq"])] = 0
    return lens


def prepare(case, seed):
    g, op, d = _gen(seed), case["op"], case["d"]
    dt = _DT[case["dtype"]]
    s = {"case": case}
    if op in ("prefill", "backward"):
        shape = (case["B"], case["H"], case["N"], d)
        s["q"], s["k"] = _randn(g, shape, dt, d ** -0.5), _randn(g, shape, dt, d ** -0.5)
        s["v"] = _randn(g, shape, dt)
        s["log_decay"] = _log_decay(case["H"], seed)
        if op == "backward":
            s["dout"] = _randn(g, shape, dt)
            s["s0"], s["ds_n"] = _state(g, (case["B"], case["H"], d, d)), _state(g, (case["B"], case["H"], d, d))
        else:
            s["s0"] = _state(g, (case["B"], case["H"], d, d)) if case["resume"] else None
    elif op == "varlen":
        lens = _lengths(case)
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        shape = (cu[-1], case["H"], d)
        s["q"], s["k"] = _randn(g, shape, dt, d ** -0.5), _randn(g, shape, dt, d ** -0.5)
        s["v"] = _randn(g, shape, dt)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["pool"] = _state(g, (4, case["H"], d, d))
        r = random.Random(int(seed) + 1)
        s["idx"] = torch.tensor([r.randint(-1, 3) for _ in lens], dtype=torch.int32, device="cuda")
        s["log_decay"] = _log_decay(case["H"], seed)
    elif op == "decode":
        shape = (case["B"], case["H"], d)
        s["q"], s["k"] = _randn(g, shape, dt, d ** -0.5), _randn(g, shape, dt, d ** -0.5)
        s["v"] = _randn(g, shape, dt)
        s["S"] = _state(g, shape + (d,)).to(_DT[case["state"]])
        s["log_decay"] = _log_decay(case["H"], seed)
    else:
        B, N, Hq, Hk = case["B"], case["N"], case["Hq"], case["Hk"]
        # one projection's output holds queries and keys side by side; the operator reads its two slices in place
        qk = _randn(g, (B, N, Hq + Hk, d), dt)
        s["q"], s["k"] = qk[:, :, :Hq].transpose(1, 2), qk[:, :, Hq:].transpose(1, 2)
        s["wq"] = ((1 + _randn(g, (d,), scale=0.1)) * d ** -0.5).to(dt)
        s["wk"] = ((1 + _randn(g, (d,), scale=0.1)) * d ** -0.5).to(dt)
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(N, device="cuda")[None]).to(torch.int32)
        if op == "norm_rope_backward":
            s["dyq"], s["dyk"] = _randn(g, (B, Hq, N, d), dt), _randn(g, (B, Hk, N, d), dt)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_scan(q, k, v, g, s0, early=False):
    """o and the last state of q, k, v [U, N, d] in fp32, log decays g [U], first state s0 [U, d, d] or None, by blocks of
    tokens.  ``early``: the state is held already decayed (it enters token 1 as it is, and leaves with one decay more)."""
    U, N, d = q.shape
    C = min(_CHUNK, max(N, 1))
    nc = max(1, -(-N // C))
    # whole blocks: zeros in front change neither the outputs behind them nor the state
    front = nc * C - N
    if front:
        z = q.new_zeros(U, front, d)
        q, k, v = torch.cat((z, q), 1), torch.cat((z, k), 1), torch.cat((z, v), 1)
    q, k, v = (x.view(U, nc, C, x.shape[-1]) for x in (q, k, v))
    i = torch.arange(C, device=q.device, dtype=torch.float64)
    g64 = g.double()[:, None]
    e = 1 if early else 0
    gap = i[:, None] - i[None, :]
    mask = torch.exp(g64[:, :, None] * gap.clamp(min=0)) * (gap >= 0)                       # [U, C, C]
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)) * mask.float()[:, None], v)
    w = torch.exp(g64 * (C - 1 - i + e)).float()                                           # [U, C]
    sums = torch.matmul((k * w[:, None, :, None]).transpose(2, 3), v)                      # [U, nc, d, d]
    c = torch.arange(nc, device=q.device, dtype=torch.float64)
    far = c[:, None] - 1 - c[None, :]
    carry = torch.exp(g64[:, :, None] * C * far.clamp(min=0)) * (far >= 0)                 # block c' -> start of block c
    starts = torch.matmul(carry.float(), sums.view(U, nc, -1)).view_as(sums)
    last = torch.matmul(torch.exp(g64 * C * (nc - 1 - c)).float()[:, None], sums.view(U, nc, -1)).view(U, *sums.shape[2:])
    if s0 is not None:
        # tokens since s0 at the start of each block (the zeros in front do not count)
        since = (c * C - front).clamp(min=0)
        first = torch.exp(g64 * since).float()[:, :, None, None] * s0[:, None]
        if front:  # block 0 is entered `front` tokens late: its rows take their distance from s0 below
            starts[:, 1:] += first[:, 1:]
        else:
            starts += first
        last = last + torch.exp(g64 * N).float()[:, :, None] * s0
    o = o + torch.matmul(q * torch.exp(g64 * (i + 1 - e)).float()[:, None, :, None], starts)
    if s0 is not None and front:
        row = torch.exp(g64 * (i + 1 - e - front).clamp(min=0)).float()[:, :, None]
        o[:, 0] += torch.matmul(q[:, 0] * row, s0)
    return o.reshape(U, nc * C, -1)[:, front:], last


def _plain_prefill(s):
    q, k, v, g = s["q"], s["k"], s["v"], s["log_decay"]
    B, H, N, d = q.shape
    flat = [x.float().reshape(B * H, N, d) for x in (q, k, v)]
    s0 = None if s["s0"] is None else s["s0"].reshape(B * H, d, d)
    o, last = _plain_scan(*flat, g.repeat(B), s0)
    return o.view(B, H, N, d).to(q.dtype), last.view(B, H, d, d)


def _plain_backward(s):
    q, k, v, do, g = s["q"], s["k"], s["v"], s["dout"], s["log_decay"]
    B, H, N, d = q.shape
    q32, k32, v32, do32 = (x.float().reshape(B * H, N, d) for x in (q, k, v, do))
    s0, ds = s["s0"].reshape(B * H, d, d), s["ds_n"].reshape(B * H, d, d)
    gu = g.repeat(B)
    dq, _ = _plain_scan(do32, v32, k32, gu, s0.transpose(1, 2))
    rq, rk, rv, rdo = (x.flip(1) for x in (q32, k32, v32, do32))
    dk, _ = _plain_scan(rv, rdo, rq, gu, ds.transpose(1, 2), early=True)
    dv, ds0 = _plain_scan(rk, rq, rdo, gu, ds, early=True)
    out = [x.reshape(B, H, N, d).to(q.dtype) for x in (dq, dk.flip(1), dv.flip(1))]
    return (*out, ds0.view(B, H, d, d))


def _plain_varlen(s):
    q, k, v, cu, g = s["q"], s["k"], s["v"], s["cu"].long(), s["log_decay"]
    T, H, d = q.shape
    n, L = cu.numel() - 1, s["case"]["max_len"]
    lens = cu[1:] - cu[:-1]
    # every sequence at the end of a row of max_len tokens (zeros in front)
    seq = torch.bucketize(torch.arange(T, device=q.device), cu[1:], right=True)
    at = seq * L + L - lens[seq] + torch.arange(T, device=q.device) - cu[seq]

    def pad(x):
        return x.new_zeros(n * L, H, d, dtype=torch.float32).index_copy_(0, at, x.float()).view(n, L, H, d) \
            .transpose(1, 2).reshape(n * H, L, d)

    init = torch.where((s["idx"] >= 0)[:, None, None, None], s["pool"][s["idx"].long().clamp(min=0)], 0.0)
    qp, gu = pad(q), g.repeat(n)
    o, last = _plain_scan(qp, pad(k), pad(v), gu, None)
    # the first state, by each token's distance from its sequence's start
    i = torch.arange(L, device=q.device) - (L - lens)[:, None] + 1                          # [n, L]
    row = torch.exp(g.double()[None, :, None] * i[:, None].clamp(min=0)).float()
    o = o.view(n, H, L, d) + torch.matmul(qp.view(n, H, L, d) * row[..., None], init)
    last = last.view(n, H, d, d) + torch.exp(g.double()[None] * lens[:, None]).float()[:, :, None, None] * init
    return o.transpose(1, 2).reshape(n * L, H, d)[at].to(q.dtype), last


def _plain_decode(s):
    q, k, v, S = (s[x].float() for x in ("q", "k", "v", "S"))
    new = S * torch.exp(s["log_decay"].double()).float()[None, :, None, None] + k[..., :, None] * v[..., None, :]
    s["S"].copy_(new)
    o = torch.matmul(q[..., None, :], s["S"].float())[..., 0, :]
    return o.to(s["q"].dtype), s["S"]


def _angles(s):
    a = s["pos"].double()[..., None] * s["inv_freq"].double()                              # [B, N, rot / 2]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


_EPS = 1e-6


def _plain_norm_rope(s):
    cos, sin = _angles(s)

    def one(x, w):
        x32 = x.float()
        y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + _EPS) * w.float()
        return _rotate(y, cos, sin, s["case"]["interleaved"]).to(x.dtype).contiguous()

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _plain_norm_rope_backward(s):
    cos, sin = _angles(s)

    def one(dy, x, w):
        x32, w32 = x.float(), w.float()
        rstd = torch.rsqrt(x32.square().mean(-1, keepdim=True) + _EPS)
        xh = x32 * rstd
        gr = _rotate(dy.float(), cos, -sin, s["case"]["interleaved"])
        dw = (gr * xh).double().sum((0, 1, 2)).float()
        wg = gr * w32
        return (rstd * (wg - xh * (wg * xh).mean(-1, keepdim=True))).to(x.dtype), dw

    (dq, dwq), (dk, dwk) = one(s["dyq"], s["q"], s["wq"]), one(s["dyk"], s["k"], s["wk"])
    return dq, dk, dwq, dwk


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import long_context_linear_b200 as la

        if op == "prefill":
            return la.prefill(s["q"], s["k"], s["v"], s["s0"], log_decay=s["log_decay"])
        if op == "varlen":
            return la.prefill_varlen(s["q"], s["k"], s["v"], s["cu"], s["pool"], s["idx"], log_decay=s["log_decay"])
        if op == "decode":
            return la.decode_step(s["q"], s["k"], s["v"], s["S"], log_decay=s["log_decay"]), s["S"]
        if op == "backward":
            return la.prefill_backward(s["q"], s["k"], s["v"], s["dout"], s["s0"], s["ds_n"], log_decay=s["log_decay"])
        if op == "norm_rope":
            return la.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["pos"], eps=_EPS,
                                   interleaved=s["case"]["interleaved"])
        return la.qk_norm_rope_backward(s["dyq"], s["dyk"], s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["pos"],
                                        eps=_EPS, interleaved=s["case"]["interleaved"])
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        return {"prefill": _plain_prefill, "varlen": _plain_varlen, "decode": _plain_decode, "backward": _plain_backward,
                "norm_rope": _plain_norm_rope, "norm_rope_backward": _plain_norm_rope_backward}[op](s)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = tf32


def work(case):
    op, d = case["op"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("prefill", "backward"):
        u = case["B"] * case["H"]
        if op == "prefill":
            return {"bytes": u * (4 * case["N"] * d * e + d * d * 4 * (2 if case["resume"] else 1)),
                    "flops": u * 4 * case["N"] * d * d}
        return {"bytes": u * (7 * case["N"] * d * e + 3 * d * d * 4), "flops": u * 12 * case["N"] * d * d}
    if op == "varlen":
        T = sum(_lengths(case))
        return {"bytes": case["H"] * (4 * T * d * e + 2 * case["n_seq"] * d * d * 4), "flops": case["H"] * 4 * T * d * d}
    if op == "decode":
        u, es = case["B"] * case["H"], 2 if case["state"] == "bf16" else 4
        return {"bytes": u * (2 * d * d * es + 4 * d * e), "flops": u * 5 * d * d}
    rows = case["B"] * case["N"] * (case["Hq"] + case["Hk"])
    if op == "norm_rope":
        return {"bytes": rows * 2 * d * e, "flops": rows * 8 * d}
    return {"bytes": rows * 3 * d * e, "flops": rows * 16 * d}


# ------------------------------------------------------------------ definitions in 64 bits

def _exact_spans(q, k, v, lam, S, early=False, span=512):
    """Over spans of tokens of [U, N, d]: o_t = sum_{s <= t} lam^(t - s) (q_t . k_s) v_s + lam^t q_t S for t = 1 ..."""
    U, N, _ = q.shape
    o = torch.empty(U, N, v.shape[-1], dtype=torch.float64, device=q.device)
    one = 0 if early else 1
    for a in range(0, N, span):
        n = min(span, N - a)
        t = torch.arange(n, device=q.device, dtype=torch.float64)
        qa, ka, va = q[:, a:a + n].double(), k[:, a:a + n].double(), v[:, a:a + n].double()
        dist = (t[:, None] - t[None, :]).clamp(min=0)
        scores = torch.einsum("utd,usd->uts", qa, ka) * torch.tril(lam ** dist)
        o[:, a:a + n] = scores @ va + (lam ** (t + one)[:, None]) * (qa @ S)
        S = lam ** n * S + (ka * lam ** (n - t - one)[:, None]).transpose(1, 2) @ va
    return o, S


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("prefill", "backward"):
        B, H, N, d = s["q"].shape
        lam = torch.exp(s["log_decay"].double()).repeat(B)[:, None, None]

        def u(x):
            return x.reshape(B * H, *x.shape[2:])

        zero = torch.zeros(B * H, d, d, dtype=torch.float64, device="cuda")
        s0 = zero if s["s0"] is None else u(s["s0"]).double()
        if op == "prefill":
            o, S = _exact_spans(u(s["q"]), u(s["k"]), u(s["v"]), lam, s0)
            return o.view(B, H, N, d), S.view(B, H, d, d)
        q, k, v, do, ds = u(s["q"]), u(s["k"]), u(s["v"]), u(s["dout"]), u(s["ds_n"]).double()
        dq, _ = _exact_spans(do, v, k, lam, s0.transpose(1, 2))
        dk, _ = _exact_spans(v.flip(1), do.flip(1), q.flip(1), lam, ds.transpose(1, 2), early=True)
        dv, ds0 = _exact_spans(k.flip(1), q.flip(1), do.flip(1), lam, ds, early=True)
        return (dq.view(B, H, N, d), dk.flip(1).view(B, H, N, d), dv.flip(1).view(B, H, N, d), ds0.view(B, H, d, d))
    if op == "varlen":
        lam = torch.exp(s["log_decay"].double())[:, None, None]
        cu, idx = s["cu"].tolist(), s["idx"].tolist()
        outs, last = [], []
        for n in range(case["n_seq"]):
            rows = slice(cu[n], cu[n + 1])
            S = s["pool"][idx[n]].double() if idx[n] >= 0 else torch.zeros_like(s["pool"][0], dtype=torch.float64)
            x = [s[a][rows].transpose(0, 1) for a in ("q", "k", "v")]
            o, S = _exact_spans(*x, lam, S)
            outs.append(o.transpose(0, 1))
            last.append(S)
        return torch.cat(outs), torch.stack(last)
    if op == "decode":
        lam = torch.exp(s["log_decay"].double())[None, :, None, None]
        S = s["S"].double() * lam + s["k"].double()[..., :, None] * s["v"].double()[..., None, :]
        if case["state"] == "bf16":
            return None  # the stored state is a rounding decision of its own, and o reads it: no 64-bit value
        return (s["q"].double()[..., None, :] @ S)[..., 0, :], S
    half = case["rot"] // 2
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                    s["pos"].double()[:, None, :, None] * s["inv_freq"].double())           # e^(i angle), [B, 1, N, half]

    def turn(x, z):
        r = x[..., :2 * half]
        pair = r.unflatten(-1, (half, 2)) if case["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
        c = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        r = c.flatten(-2) if case["interleaved"] else c.transpose(-1, -2).flatten(-2)
        return torch.cat((r, x[..., 2 * half:]), -1)

    def norm(x, w):
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) * w

    q, k, wq, wk = (s[a].double() for a in ("q", "k", "wq", "wk"))
    if op == "norm_rope":
        return turn(norm(q, wq), z), turn(norm(k, wk), z)
    got = []
    for x, w, dy in ((q, wq, s["dyq"]), (k, wk, s["dyk"])):
        x, w = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
        got.append(torch.autograd.grad(norm(x, w), (x, w), turn(dy.double(), z.conj())))
    return got[0][0], got[1][0], got[0][1], got[1][1]
