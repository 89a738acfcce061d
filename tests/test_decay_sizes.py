"""The Python size queries cover the calls with a decay, so that a caller's own
workspace is the one that is used (the queries' values on the CPU, their use on a
GPU)."""
import pytest
import torch

import long_context_linear_b200 as la
from long_context_linear_b200 import _abi

B16, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 76, 700, 128), (4, 32, 8192, 128), (1, 6, 20011, 64), (1, 2, 256, 64), (1, 3, 777, 64), (1, 1, 1, 128)]


@pytest.mark.parametrize("dt", [B16, F32])
@pytest.mark.parametrize("B,H,N,d", SIZES)
def test_queries(B, H, N, d, dt):
    args = (B, H, N, d, d, _abi.LA_BF16 if dt == B16 else _abi.LA_FP32)
    assert la.prefill_workspace_size(B, H, N, d, dt, decay=True) == la.lib.la_prefill_decay_workspace_size(*args)
    assert la.prefill_workspace_size(B, H, N, d, dt) == la.lib.la_prefill_workspace_size(*args)
    assert la.prefill_backward_workspace_size(B, H, N, d, dt) == la.lib.la_prefill_backward_workspace_size(*args)
    assert la.prefill_backward_workspace_size(B, H, N, d, dt, decay=True) == \
        la.lib.la_prefill_decay_backward_workspace_size(*args)
    # (a packed call needs the same with a decay as without)
    assert la.prefill_varlen_workspace_size(B, N, H, d, dt) == \
        la.lib.la_prefill_varlen_decay_workspace_size(B, N, H, *args[3:])


def test_decay_takes_no_feature_map():
    with pytest.raises(ValueError):
        la.prefill_workspace_size(1, 1, 128, 128, B16, "relu", decay=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [B16, F32])
@pytest.mark.parametrize("B,H,N,d", SIZES)
def test_a_workspace_of_that_size_is_used(B, H, N, d, dt):
    """No allocation but the outputs', and the results of a call without one."""
    q, k, v, do = (torch.randn(B, H, N, d, device="cuda").to(dt) for _ in range(4))
    g = -torch.rand(H, device="cuda")
    out, s_out = torch.empty_like(v), torch.empty(B, H, d, d, device="cuda")
    ws = torch.empty(la.prefill_workspace_size(B, H, N, d, dt, decay=True), dtype=torch.uint8, device="cuda")
    want = la.prefill(q, k, v, log_decay=g)
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    la.prefill(q, k, v, log_decay=g, out=out, s_out=s_out, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert torch.equal(out, want[0]) and torch.equal(s_out, want[1])
    ws = torch.empty(la.prefill_backward_workspace_size(B, H, N, d, dt, decay=True), dtype=torch.uint8, device="cuda")
    want = la.prefill_backward(q, k, v, do, log_decay=g)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    got = la.prefill_backward(q, k, v, do, log_decay=g, workspace=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before + 4  # dq, dk, dv, dS_0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
