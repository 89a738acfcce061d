"""The decayed prefill in a context that has fewer SMs than the device: the schedule
whose CTAs hand states on to one another needs all of them resident, and where they
are not the units run whole, with the same bits."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import long_context_linear_b200 as la
    return la


@pytest.mark.skipif(not torch.cuda.green_contexts.SUPPORTED, reason="no contexts of some of the SMs")
@pytest.mark.parametrize("d,H", [(128, 76), (64, 149)])
def test_same_bits(la, d, H):
    N = 900
    q, k, v = (t.cuda() for t in synth.dense(1, H, N, d, "bf16", seed=3))
    g = -torch.rand(H, device="cuda")
    assert la.prefill_workspace_size(1, H, N, d, torch.bfloat16, decay=True) > 0
    want = la.prefill(q, k, v, log_decay=g)
    grads = la.prefill_backward(q, k, v, want[0], None, want[1], log_decay=g)
    torch.cuda.synchronize()
    few = torch.cuda.GreenContext.create(num_sms=16, device_id=torch.cuda.current_device())
    few.set_context()
    try:
        got = la.prefill(q, k, v, log_decay=g)
        dgot = la.prefill_backward(q, k, v, want[0], None, want[1], log_decay=g)
        torch.cuda.synchronize()
    finally:
        few.pop_context()
    for a, b in zip((*got, *dgot), (*want, *grads)):
        assert torch.equal(a, b)
    assert la.device_status() == 0
