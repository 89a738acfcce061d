"""Callers' workspaces: a buffer that the kernels could not write (on the host, on
another device, a view that is larger than its memory) is refused before any
launch.  The check itself on the CPU, the calls that use it on a GPU."""
import pytest
import torch

import long_context_linear_b200 as la

DEV = torch.device("cuda", 0)
BAD = [torch.empty(1 << 10, dtype=torch.uint8),                       # on the host
       torch.empty(1 << 10, dtype=torch.uint8, device="meta"),
       [0] * 1024]


@pytest.mark.parametrize("need", [0, 1, 1 << 10, 1 << 20])
@pytest.mark.parametrize("bad", range(len(BAD)))
def test_refused(bad, need):
    with pytest.raises((ValueError, TypeError)):
        la._workspace(BAD[bad], need, DEV)


def test_none_needed():
    assert la._workspace(None, 0, DEV) == (None, 0)


def test_sizes():
    cpu = torch.device("cpu")
    ws, n = la._workspace(torch.empty(100, dtype=torch.float32), 400, cpu)
    assert n == 400 and ws.dtype == torch.float32
    for given in (None, torch.empty(100)):
        ws, n = la._workspace(given, 401, cpu)  # none given, or too small: a new one
        assert n == 401 == ws.numel() and ws.device == cpu
    for view in (torch.empty(1).expand(1000), torch.empty(64, 64).t()[:, :32], torch.empty(64)[::2]):
        with pytest.raises(ValueError):
            la._workspace(view, 16, cpu)


@pytest.mark.gpu
@pytest.mark.parametrize("ws", [torch.empty(1 << 26, dtype=torch.uint8), "expanded"])
def test_calls_refuse(ws):
    if isinstance(ws, str):
        ws = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 26)
    x = torch.zeros(1, 2, 4096, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(4096, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 4096], dtype=torch.int32, device="cuda")
    g, w = torch.zeros(2, device="cuda"), torch.ones(64, device="cuda")
    h = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    for call in (lambda: la.prefill(x, x, x, workspace=ws), lambda: la.prefill(x, x, x, log_decay=g, workspace=ws),
                 lambda: la.prefill_varlen(p, p, p, cu, workspace=ws),
                 lambda: la.prefill_varlen(p, p, p, cu, log_decay=g, workspace=ws),
                 lambda: la.prefill_backward(x, x, x, x, workspace=ws),
                 lambda: la.prefill_backward(x, x, x, x, log_decay=g, workspace=ws),
                 lambda: la.qk_norm_rope_backward(x, x, x, x, w, w, workspace=ws),
                 lambda: la.prefill_host(h, h, h, workspace=ws)):
        with pytest.raises(ValueError, match="workspace"):
            call()
