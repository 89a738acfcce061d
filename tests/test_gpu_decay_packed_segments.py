"""States carried from segment to segment of packed sequences, with decays that a
segment leaves part of (exp(len g) between 0.2 and 0.98): a factor of a wrong length
shows at 5e-6.  Tolerances as in test_gpu_decay.py (sqrt(5000) 2^-24 = 4.2e-6)."""
import numpy as np
import pytest
import torch

import synth
from oracle import decay as od
from tests.parity import assert_state, assert_varlen_out

pytestmark = pytest.mark.gpu
STATE = 5e-6


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


def check(la, dtype, d, lens, g, seed):
    H = len(g)
    cu = synth.cu_seqlens(lens)
    q, k, v = synth.qkv((int(cu[-1]), H, d), d, dtype, seed=seed)
    pool = synth.outer_product_state(3 * H, d, d, [64] * (3 * H), seed=seed + 1).view(3, H, d, d) * 4
    idx = torch.tensor([(i % 4) - 1 for i in range(len(lens), 0, -1)], dtype=torch.int32)
    o, s = la.prefill_varlen(*(t.cuda() for t in (q, k, v, cu, pool, idx)), log_decay=g.cuda())
    torch.cuda.synchronize()
    assert la.device_status() == 0
    ro, rs = od.varlen(q, k, v, cu, g, pool, idx)
    assert_varlen_out(o.cpu(), ro, cu, q.dtype)
    assert_state(s.cpu(), rs, 2, tol=STATE)
    return q, k, v, cu, pool, idx, rs


KINDS = [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)]


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("segments", ["1", "2", "3", "9"])
def test_given_segments(la, monkeypatch, dtype, d, segments):
    monkeypatch.setenv("LA_PREFILL_SEGMENTS", segments)
    check(la, dtype, d, [1500, 3, 0, 700, 261], torch.tensor([-1e-4, -1e-3, -5e-3]), seed=31)


@pytest.mark.parametrize("dtype,d", KINDS)
@pytest.mark.parametrize("lens", [[5000, 77, 2100], [2049], [0, 4097, 1]])
def test_segments_of_the_library_s_choice(la, dtype, d, lens):
    """Few heads and 2048 tokens or more: cut into segments of at least 1024."""
    base = 256 * -(-len(lens) * 4 // 256)
    state = 2 * d * d * 4
    assert la.prefill_varlen_workspace_size(len(lens), sum(lens), 2, d, synth.torch_dtype(dtype)) >= base + state
    check(la, dtype, d, lens, torch.tensor([-1e-4, -1e-3]), seed=32)


def test_a_wrong_length_would_show():
    """The oracle with a segment's factor one token short, or the tail's: far outside the bar."""
    d, lens, seg = 64, [1500], 256
    g = torch.tensor([-1e-4, -1e-3, -5e-3])
    q, k, v = synth.qkv((1500, 3, d), d, "bf16", seed=31)
    want = od.varlen(q, k, v, [0, 1500], g)[1]

    def carried(length):
        S = np.zeros((1, 3, d, d))
        for a in range(0, 1500, seg):
            n = min(seg, 1500 - a)
            own = od.varlen(q[a:a + n], k[a:a + n], v[a:a + n], [0, n], g)[1]
            S = np.exp(g.double().numpy() * (n if n < seg else length))[:, None, None] * S + own
        return S

    rel = [(np.linalg.norm(carried(n) - want, axis=(2, 3)) / np.linalg.norm(want, axis=(2, 3))) for n in (seg, seg - 1, 1500 % seg)]
    assert rel[0].max() < 1e-12 and min(rel[1].min(), rel[2].min()) > 10 * STATE
