"""Refusals of the decayed attention's and the norm's entry points, on the host
(CPU: every call fails before the device is touched)."""
import ctypes

import pytest

FAKE = 1 << 20  # a 16-byte aligned non-null "device pointer"; never dereferenced on these paths


@pytest.fixture(scope="module")
def abi():
    from long_context_linear_b200 import _abi
    return _abi


def _prefill(abi, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, s0=None, s_out=None, g=FAKE, B=1, H=1, N=16, dk=128, dv=128, dt=0, chunk=0)
    a.update(kw)
    return abi.lib.la_prefill_decay(a["q"], a["k"], a["v"], a["o"], a["s0"], a["s_out"], a["g"], a["B"], a["H"], a["N"],
                                    a["dk"], a["dv"], a["dt"], a["chunk"], None, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), 1), (dict(dk=96, dv=96), 2), (dict(dk=128, dv=64), 2), (dict(dt=7), 1), (dict(N=-1), 1),
    (dict(H=-1), 1), (dict(q=None), 1), (dict(o=FAKE + 8), 1), (dict(s0=FAKE + 4), 1), (dict(chunk=48), 2),
])
def test_prefill_decay_refuses(abi, kw, status):
    assert _prefill(abi, **kw) == status
    assert abi.lib.la_last_error()


def test_prefill_decay_of_nothing_is_ok(abi):
    assert _prefill(abi, B=0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), 1), (dict(dk=32, dv=32), 2), (dict(cu=None), 1), (dict(n_seq=-1), 1), (dict(T=-1), 1),
    (dict(q=None), 1), (dict(pool=None, idx=FAKE), 1), (dict(k=FAKE + 2), 1),
])
def test_varlen_decay_refuses(abi, kw, status):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, cu=FAKE, n_seq=2, T=16, pool=None, n_pool=0, idx=None, g=FAKE, H=1, dk=128,
             dv=128, dt=1)
    a.update(kw)
    st = abi.lib.la_prefill_varlen_decay(a["q"], a["k"], a["v"], a["o"], a["cu"], a["n_seq"], a["T"], a["pool"],
                                         a["n_pool"], a["idx"], None, a["g"], a["H"], a["dk"], a["dv"], a["dt"], 0, None,
                                         0, None)
    assert st == status


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), 1), (dict(dk=32, dv=32), 2), (dict(sdt=9), 1), (dict(dt=1, sdt=1), 2), (dict(S=None), 1),
    (dict(S=FAKE + 4), 1), (dict(B=-1), 1),
])
def test_decode_decay_refuses(abi, kw, status):
    a = dict(S=FAKE, g=FAKE, B=1, H=1, dk=128, dv=128, dt=0, sdt=0)
    a.update(kw)
    assert abi.lib.la_decode_step_decay(FAKE, FAKE, FAKE, FAKE, a["S"], a["g"], a["B"], a["H"], a["dk"], a["dv"],
                                        a["dt"], a["sdt"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), 1), (dict(dk=32, dv=32), 2), (dict(dq=None), 1), (dict(ds0=FAKE + 4), 1), (dict(N=-1), 1),
])
def test_backward_decay_refuses(abi, kw, status):
    a = dict(g=FAKE, dq=FAKE, ds0=FAKE, B=1, H=1, N=8, dk=128, dv=128)
    a.update(kw)
    assert abi.lib.la_prefill_decay_backward(FAKE, FAKE, FAKE, FAKE, None, None, a["g"], a["dq"], FAKE, FAKE, a["ds0"],
                                             a["B"], a["H"], a["N"], a["dk"], a["dv"], 0, None, 0, None) == status


def _view(abi, p=FAKE, sb=4096, sh=128, sn=1024):
    return ctypes.byref(abi.View(p, sb, sh, sn))


def _norm_rope(abi, backward=False, **kw):
    a = dict(q={}, k={}, qo={}, ko={}, wq=FAKE, wk=FAKE, f=FAKE, pos=FAKE, pos64=0, B=2, N=4, Hq=2, Hk=1, d=128, rot=128,
             eps=1e-6, dt=0, wdt=0, ws=FAKE, wsb=1 << 30, gw=FAKE)
    a.update(kw)
    views = [None if a[x] is None else _view(abi, **a[x]) for x in ("q", "k", "qo", "ko")]
    tail = (a["B"], a["N"], a["Hq"], a["Hk"], a["d"], a["rot"], a["eps"], 0, a["dt"], a["wdt"])
    mid = (a["wq"], a["wk"], a["f"], a["pos"], a["pos64"], 4, 1)
    if backward:
        return abi.lib.la_qk_norm_rope_backward(*views[2:], *views[:2], *mid, *views[:2], a["gw"], a["gw"], *tail, a["ws"],
                                                a["wsb"], None)
    return abi.lib.la_qk_norm_rope(*views, *mid, *tail, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(ko=None), 1), (dict(q=dict(p=None)), 1), (dict(q=dict(p=FAKE + 8)), 1),
    (dict(k=dict(sn=1025)), 1), (dict(qo=dict(sh=4)), 1), (dict(wq=None), 1), (dict(wk=FAKE + 4), 1), (dict(f=None), 1),
    (dict(f=FAKE + 2), 1), (dict(pos=FAKE + 4, pos64=1), 1), (dict(B=-1), 1), (dict(N=-1), 1), (dict(Hk=-1), 1),
    (dict(d=96), 2), (dict(rot=24), 2), (dict(rot=144), 2), (dict(rot=-16), 2), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(dt=5), 1), (dict(dt=1, wdt=0), 2),
])
def test_norm_rope_refuses(abi, kw, status, backward):
    assert _norm_rope(abi, backward, **kw) == status
    assert abi.lib.la_last_error()


@pytest.mark.parametrize("view", [dict(sb=0), dict(sh=0), dict(sn=0)])
def test_norm_rope_refuses_outputs_that_share_memory(abi, view):
    assert _norm_rope(abi, qo=view) == 1 and b"q_out" in abi.lib.la_last_error()
    if "sh" not in view:  # (one key head: its stride says nothing)
        assert _norm_rope(abi, ko=view) == 1 and b"k_out" in abi.lib.la_last_error()
    assert _norm_rope(abi, True, q=view) == 1 and b"dq" in abi.lib.la_last_error()


@pytest.mark.parametrize("kw", [dict(ws=None), dict(ws=FAKE + 8), dict(wsb=64), dict(gw=FAKE + 2)])
def test_norm_rope_backward_refuses_its_own(abi, kw):
    assert _norm_rope(abi, True, **kw) == 1


def test_norm_rope_of_nothing_is_ok(abi):
    assert _norm_rope(abi, B=0) == 0
    assert _norm_rope(abi, Hq=0, Hk=0) == 0


def test_python_wrappers_refuse_host_tensors():
    import torch

    import long_context_linear_b200 as la
    x = torch.zeros(1, 2, 4, 128)
    g = torch.zeros(2)
    with pytest.raises(ValueError):
        la.prefill(x, x, x, log_decay=g)
    with pytest.raises(ValueError):
        la.prefill_backward(x, x, x, x, log_decay=g)
    with pytest.raises(ValueError):
        la.decode_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], torch.zeros(1, 2, 128, 128), log_decay=g)
    with pytest.raises(ValueError):
        la.qk_norm_rope(x, x, torch.ones(128), torch.ones(128))
