"""Causal linear attention (Lightning Attention, phi = identity) for B200.

Python binding of the C ABI in ``include/la.h``: every function below only
checks and marshals arguments (torch tensors -> device pointers, the current
CUDA stream) and calls the CUDA library; all computation runs in its kernels.

    S_t = S_{t-1} + k_t (x) v_t,   o_t = q_t S_t

(page "MiniMax-M1で理解する…" (zenn.dev), section "線形アテンションの数学的基礎";
tiled as on page "MiniMax: «Почему M2 в итоге стала моделью с полным
вниманием?»", section 1, glossary entry "Lightning Attention").  With ``log_decay`` the state decays
between tokens, S_t = exp(log_decay[h]) S_{t-1} + k_t (x) v_t for head h.
``qk_norm_rope`` forms the queries and keys from a projection's output: the norm
of every head and the rotation by the token's position.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _abi
from ._abi import LAError, lib

__all__ = ["prefill", "prefill_host", "prefill_varlen", "prefill_varlen_noalloc", "prefill_backward", "decode_step",
           "decode_verify",
           "decode_commit", "qk_norm_rope", "qk_norm_rope_backward",
           "device_status", "LAError",
           "lib", "prefill_workspace_size", "prefill_varlen_workspace_size", "prefill_backward_workspace_size"]

_DT = {torch.bfloat16: _abi.LA_BF16, torch.float32: _abi.LA_FP32}
PHI = {"identity": _abi.LA_PHI_IDENTITY, "elu1": _abi.LA_PHI_ELU1, "relu": _abi.LA_PHI_RELU}


def _phi_code(phi: str) -> int:
    if phi not in PHI:
        raise ValueError(f"unknown feature map {phi!r}; one of {sorted(PHI)}")
    return PHI[phi]


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")
    return _DT[t.dtype]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device: torch.device):
    # the handle alone, without a stream object around it (2 us of a call's 17)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device.index is None else device.index)


class _Here:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return None


_HERE = _Here()


def _on(device: torch.device):
    """The tensors' device made current for a call (nothing to do, and no time spent, when it already is)."""
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _need(t: torch.Tensor, name: str, dtype=None, device=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _workspace(workspace: Optional[torch.Tensor], need: int, device: torch.device):
    """A call's workspace and its bytes: the given one if it has `need` bytes, else a new one (None if need is 0).
    The kernels write to a given one, so it has to be memory of the tensors' device."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError(f"workspace must be a tensor, got {type(workspace).__name__}")
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, expected {device}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        size = workspace.numel() * workspace.element_size()
        if size >= need:
            return workspace, size
    return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)


def _check_decay(log_decay: torch.Tensor, H: int, device, phi: str = "identity"):
    """log_decay: fp32 [H] on the tensors' device, without a feature map."""
    _need(log_decay, "log_decay", torch.float32, device)
    if tuple(log_decay.shape) != (H,):
        raise ValueError(f"log_decay must be [H] = [{H}], got {tuple(log_decay.shape)}")
    if phi != "identity":
        raise ValueError("log_decay needs phi='identity'")


def _need_host(t: torch.Tensor, name: str, dtype=None):
    if t.device.type != "cpu":
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def prefill_workspace_size(B: int, H: int, N: int, d: int, dtype: torch.dtype, phi: str = "identity", *,
                           decay: bool = False) -> int:
    """Bytes of workspace that ``prefill`` asks for (decay: with log_decay)."""
    if decay:
        if phi != "identity":
            raise ValueError("a decay needs phi='identity'")
        return int(lib.la_prefill_decay_workspace_size(B, H, N, d, d, _DT[dtype]))
    return int(lib.la_prefill_workspace_size_ex(B, H, N, d, d, _DT[dtype], _phi_code(phi)))


def prefill_backward_workspace_size(B: int, H: int, N: int, d: int, dtype: torch.dtype, *, decay: bool = False) -> int:
    """Bytes of workspace that ``prefill_backward`` asks for (decay: with log_decay)."""
    return int((lib.la_prefill_decay_backward_workspace_size if decay else lib.la_prefill_backward_workspace_size)(
        B, H, N, d, d, _DT[dtype]))


def prefill_varlen_workspace_size(n_seq: int, T: int, H: int, d: int, dtype: torch.dtype,
                                  phi: str = "identity") -> int:
    """Bytes of workspace that ``prefill_varlen`` asks for, with or without log_decay."""
    return int(lib.la_prefill_varlen_workspace_size_ex(n_seq, T, H, d, d, _DT[dtype], _phi_code(phi)))


def prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, s0: Optional[torch.Tensor] = None, *,
            chunk: int = 0, out: Optional[torch.Tensor] = None, s_out: Optional[torch.Tensor] = None,
            return_state: bool = True, workspace: Optional[torch.Tensor] = None, phi: str = "identity",
            log_decay: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Dense prefill over q, k, v of shape [B, H, N, d]; returns (O, S_N).

    s0 (fp32 [B, H, d, d]) is the state before the first token (zero if None);
    phi ("identity", "elu1", "relu") is the feature map on q and k.  log_decay
    (fp32 [H], values <= 0): S_t = exp(log_decay[h]) S_{t-1} + k_t (x) v_t
    (identity feature map only).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    if q.dim() != 4 or k.shape != q.shape or v.shape[:3] != q.shape[:3]:
        raise ValueError("q, k must be [B, H, N, dk] and v [B, H, N, dv]")
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, device=q.device)
    _need(out, "out", q.dtype, q.device)
    if s0 is not None:
        _need(s0, "s0", torch.float32, q.device)
        if tuple(s0.shape) != (B, H, dk, dv):
            raise ValueError("s0 must be [B, H, dk, dv]")
    if s_out is None and return_state:
        s_out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if s_out is not None:
        _need(s_out, "s_out", torch.float32, q.device)
    if log_decay is not None:
        _check_decay(log_decay, H, q.device, phi)
        if tuple(out.shape) != (B, H, N, dv) or (s_out is not None and tuple(s_out.shape) != (B, H, dk, dv)):
            raise ValueError("out must be [B, H, N, dv] and s_out [B, H, dk, dv]")
    need = int(lib.la_prefill_workspace_size_ex(B, H, N, dk, dv, dt, _phi_code(phi)) if log_decay is None
               else lib.la_prefill_decay_workspace_size(B, H, N, dk, dv, dt))
    workspace, ws_bytes = _workspace(workspace, need, q.device)
    with _on(q.device):
        if log_decay is not None:
            _abi.check(lib.la_prefill_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(s0), _ptr(s_out),
                                            _ptr(log_decay), B, H, N, dk, dv, dt, chunk, _ptr(workspace), ws_bytes,
                                            _stream(q.device)), "la_prefill_decay")
            return out, s_out
        _abi.check(lib.la_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(s0), _ptr(s_out),
                                     B, H, N, dk, dv, dt, chunk, _phi_code(phi), _ptr(workspace), ws_bytes,
                                     _stream(q.device)),
                   "la_prefill_ex")
    return out, s_out


def prefill_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, s0: Optional[torch.Tensor] = None, *,
                 group: int = 8, out: Optional[torch.Tensor] = None, s_out: Optional[torch.Tensor] = None,
                 return_state: bool = True, workspace: Optional[torch.Tensor] = None,
                 device: Optional[torch.device] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``prefill`` on host tensors (page-locked for overlap): q, k, v [B, H, N, d]
    and s0 [B, H, d, d] fp32 on the CPU; returns host (O, S_N).

    Groups of ``group`` (batch, head) units are copied in, computed and copied
    out on overlapping streams of ``device`` (default: the current CUDA
    device).  Asynchronous: synchronise that device's current stream before
    reading the results.
    """
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_host(t, n, q.dtype)
    if q.dim() != 4 or k.shape != q.shape or v.shape[:3] != q.shape[:3]:
        raise ValueError("q, k must be [B, H, N, dk] and v [B, H, N, dv]")
    B, H, N, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    pin = torch.cuda.is_available()
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, pin_memory=pin)
    _need_host(out, "out", q.dtype)
    if s0 is not None:
        _need_host(s0, "s0", torch.float32)
        if tuple(s0.shape) != (B, H, dk, dv):
            raise ValueError("s0 must be [B, H, dk, dv]")
    if s_out is None and return_state:
        s_out = torch.empty((B, H, dk, dv), dtype=torch.float32, pin_memory=pin)
    if s_out is not None:
        _need_host(s_out, "s_out", torch.float32)
    need = int(lib.la_prefill_host_workspace_size(B, H, N, dk, dv, dt, group))
    workspace, ws_bytes = _workspace(workspace, max(need, 1), dev)
    with torch.cuda.device(dev):
        _abi.check(lib.la_prefill_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(s0), _ptr(s_out), B, H, N, dk, dv,
                                       dt, group, _ptr(workspace), ws_bytes, _stream(dev)), "la_prefill_host")
    return out, s_out


def prefill_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dout: torch.Tensor,
                     s0: Optional[torch.Tensor] = None, ds_n: Optional[torch.Tensor] = None, *,
                     need_ds0: bool = True, workspace: Optional[torch.Tensor] = None,
                     log_decay: Optional[torch.Tensor] = None):
    """Gradients of ``prefill`` for dL/dO = dout and dL/dS_N = ds_n (zero if None).

    q, k, v, dout: [B, H, N, d]; s0, ds_n: fp32 [B, H, d, d] or None; log_decay
    as given to ``prefill`` (a constant: it has no gradient).
    Returns (dq, dk, dv, ds0) with dq, dk, dv in the input dtype and ds0 fp32
    (None unless need_ds0).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, n, q.dtype, q.device)
    if q.dim() != 4 or k.shape != q.shape or v.shape != q.shape or dout.shape != v.shape:
        raise ValueError("q, k, v, dout must all be [B, H, N, d]")
    B, H, N, d = q.shape
    for t, n in ((s0, "s0"), (ds_n, "ds_n")):
        if t is not None:
            _need(t, n, torch.float32, q.device)
            if tuple(t.shape) != (B, H, d, d):
                raise ValueError(f"{n} must be [B, H, d, d]")
    if log_decay is not None:
        _check_decay(log_decay, H, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ds0 = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device) if need_ds0 else None
    need = int((lib.la_prefill_backward_workspace_size if log_decay is None
                else lib.la_prefill_decay_backward_workspace_size)(B, H, N, d, d, _dtype_code(q)))
    workspace, ws_bytes = _workspace(workspace, need, q.device)
    with _on(q.device):
        if log_decay is not None:
            _abi.check(lib.la_prefill_decay_backward(
                _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(s0), _ptr(ds_n), _ptr(log_decay), _ptr(dq), _ptr(dk),
                _ptr(dv), _ptr(ds0), B, H, N, d, d, _dtype_code(q), _ptr(workspace), ws_bytes, _stream(q.device)),
                "la_prefill_decay_backward")
            return dq, dk, dv, ds0
        _abi.check(lib.la_prefill_backward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(s0), _ptr(ds_n), _ptr(dq),
                                              _ptr(dk), _ptr(dv), _ptr(ds0), B, H, N, d, d, _dtype_code(q),
                                              _ptr(workspace), ws_bytes, _stream(q.device)), "la_prefill_backward_ex")
    return dq, dk, dv, ds0


def _check_packed(q, k, v, cu_seqlens, state_pool, init_idx, out, s_out):
    """Device, dtype, contiguity and shape checks of a packed ragged batch;
    returns (T, H, dk, dv, n_seq, n_pool).  Run before any launch, so that a
    wrongly sized buffer never reaches a kernel."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    _need(cu_seqlens, "cu_seqlens", torch.int32, q.device)
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[:2] != q.shape[:2]:
        raise ValueError("q, k must be [T, H, dk] and v [T, H, dv]")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    T, H, dk = q.shape
    dv = v.shape[-1]
    n_seq = cu_seqlens.numel() - 1
    if out is not None:
        _need(out, "out", q.dtype, q.device)
        if tuple(out.shape) != (T, H, dv):
            raise ValueError(f"out must be [T, H, dv] = {(T, H, dv)}, got {tuple(out.shape)}")
    n_pool = 0
    if state_pool is not None:
        _need(state_pool, "state_pool", torch.float32, q.device)
        if state_pool.dim() != 4 or tuple(state_pool.shape[1:]) != (H, dk, dv):
            raise ValueError("state_pool must be [n_pool, H, dk, dv]")
        n_pool = state_pool.shape[0]
    if init_idx is not None:
        _need(init_idx, "init_idx", torch.int32, q.device)
        if init_idx.numel() != n_seq:
            raise ValueError("init_idx must have n_seq entries")
    if s_out is not None:
        _need(s_out, "s_out", torch.float32, q.device)
        if tuple(s_out.shape) != (n_seq, H, dk, dv):
            raise ValueError(f"s_out must be [n_seq, H, dk, dv] = {(n_seq, H, dk, dv)}, got {tuple(s_out.shape)}")
    return T, H, dk, dv, n_seq, n_pool


def prefill_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                   state_pool: Optional[torch.Tensor] = None, init_idx: Optional[torch.Tensor] = None, *,
                   chunk: int = 0, out: Optional[torch.Tensor] = None, s_out: Optional[torch.Tensor] = None,
                   return_state: bool = True, workspace: Optional[torch.Tensor] = None, phi: str = "identity",
                   log_decay: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Packed ragged prefill: q, k [T, H, d], v [T, H, d], cu_seqlens int32 [n_seq + 1].

    Sequence n starts from state_pool[init_idx[n]] when init_idx[n] >= 0;
    phi is the feature map on q and k, log_decay (fp32 [H], <= 0) the decay per
    head (identity feature map only).  Returns (O [T, H, d], S [n_seq, H, d, d]);
    rows of O behind the last sequence are left as they were.
    """
    T, H, dk, dv, n_seq, n_pool = _check_packed(q, k, v, cu_seqlens, state_pool, init_idx, out, s_out)
    dt = _dtype_code(q)
    if log_decay is not None:
        _check_decay(log_decay, H, q.device, phi)
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=q.device)
    if s_out is None and return_state:
        s_out = torch.empty((max(n_seq, 0), H, dk, dv), dtype=torch.float32, device=q.device)
    need = int(lib.la_prefill_varlen_workspace_size_ex(n_seq, T, H, dk, dv, dt, _phi_code(phi)))
    workspace, ws_bytes = _workspace(workspace, need, q.device)
    with _on(q.device):
        if log_decay is not None:
            _abi.check(lib.la_prefill_varlen_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(cu_seqlens), n_seq, T,
                                                   _ptr(state_pool), n_pool, _ptr(init_idx), _ptr(s_out),
                                                   _ptr(log_decay), H, dk, dv, dt, chunk, _ptr(workspace), ws_bytes,
                                                   _stream(q.device)), "la_prefill_varlen_decay")
            return out, s_out
        _abi.check(lib.la_prefill_varlen_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(cu_seqlens), n_seq, T,
                                            _ptr(state_pool), n_pool, _ptr(init_idx), _ptr(s_out), H, dk, dv, dt,
                                            chunk, _phi_code(phi), _ptr(workspace), ws_bytes, _stream(q.device)),
                   "la_prefill_varlen_ex")
    return out, s_out


def prefill_varlen_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                           state_pool: Optional[torch.Tensor] = None, init_idx: Optional[torch.Tensor] = None, *,
                           out: torch.Tensor, s_out: Optional[torch.Tensor] = None, chunk: int = 0) -> None:
    """prefill_varlen for callers that cannot allocate device memory.

    The caller passes every output buffer; the library uses its built-in
    scratch (at most ``_abi.NOALLOC_MAX_SEQS`` sequences per call) instead of a
    workspace.  Calls share that scratch: order them on one stream.  With no
    workspace the call never cuts sequences into segments, so batches of a few
    long sequences run one CTA per (sequence, head, value slice); the feature
    map is the identity.
    """
    if out is None:
        raise ValueError("out is required: this call allocates nothing")
    T, H, dk, dv, n_seq, n_pool = _check_packed(q, k, v, cu_seqlens, state_pool, init_idx, out, s_out)
    with torch.cuda.device(q.device):
        _abi.check(lib.la_prefill_varlen_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(cu_seqlens), n_seq, T,
                                                 _ptr(state_pool), n_pool, _ptr(init_idx), _ptr(s_out), H, dk, dv,
                                                 _dtype_code(q), chunk, _stream(q.device)),
                   "la_prefill_varlen_noalloc")


_STATE_DT = {torch.float32: _abi.LA_STATE_FP32, torch.bfloat16: _abi.LA_STATE_BF16,
             torch.float16: _abi.LA_STATE_FP16, torch.float8_e4m3fn: _abi.LA_STATE_FP8_E4M3,
             torch.float8_e5m2: _abi.LA_STATE_FP8_E5M2}


def decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, S: torch.Tensor, *,
                out: Optional[torch.Tensor] = None, phi: str = "identity",
                log_decay: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token per (batch, head): S <- S + k (x) v in place, returns o = q S.

    With log_decay (fp32 [H], values <= 0; identity feature map only)
    S <- exp(log_decay[h]) S + k (x) v.

    q, k, v: [B, H, d]; S: [B, H, d, d] in fp32, or in bf16 / fp16 /
    float8_e4m3fn / float8_e5m2 (state stored in low precision, updated in fp32
    and rounded to nearest even, the 8-bit formats saturating at their largest
    finite value; needs bf16 q, k, v).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    if S.dtype not in _STATE_DT:
        raise TypeError(f"S must be float32, bfloat16, float16, float8_e4m3fn or float8_e5m2, got {S.dtype}")
    _need(S, "S", S.dtype, q.device)
    if q.dim() != 3 or k.shape != q.shape or v.shape[:2] != q.shape[:2]:
        raise ValueError("q, k must be [B, H, dk] and v [B, H, dv]")
    B, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(S.shape) != (B, H, dk, dv):
        raise ValueError("S must be [B, H, dk, dv]")
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    _need(out, "out", q.dtype, q.device)
    if log_decay is not None:
        _check_decay(log_decay, H, q.device, phi)
        if tuple(out.shape) != (B, H, dv):
            raise ValueError("out must be [B, H, dv]")
        with _on(q.device):
            _abi.check(lib.la_decode_step_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), _ptr(log_decay), B, H,
                                                dk, dv, _dtype_code(q), _STATE_DT[S.dtype], _stream(q.device)),
                       "la_decode_step_decay")
        return out
    with torch.cuda.device(q.device):
        _abi.check(lib.la_decode_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), B, H, dk, dv,
                                         _dtype_code(q), _STATE_DT[S.dtype], _phi_code(phi), _stream(q.device)),
                   "la_decode_step_ex")
    return out


def decode_verify(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, S: torch.Tensor, *,
                  out: Optional[torch.Tensor] = None, phi: str = "identity") -> torch.Tensor:
    """Outputs for m draft tokens per (batch, head) without changing S.

    q, k, v: [B, H, m, d] (1 <= m <= 16); S: fp32 [B, H, d, d] (read only).
    Returns o [B, H, m, d] with o_t = q_t (S + sum_{s<=t} k_s (x) v_s).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype, q.device)
    _need(S, "S", torch.float32, q.device)
    if q.dim() != 4 or k.shape != q.shape or v.shape[:3] != q.shape[:3]:
        raise ValueError("q, k must be [B, H, m, dk] and v [B, H, m, dv]")
    B, H, m, dk = q.shape
    dv = v.shape[-1]
    if tuple(S.shape) != (B, H, dk, dv):
        raise ValueError("S must be [B, H, dk, dv]")
    if out is None:
        out = torch.empty((B, H, m, dv), dtype=q.dtype, device=q.device)
    _need(out, "out", q.dtype, q.device)
    with torch.cuda.device(q.device):
        _abi.check(lib.la_decode_verify(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(S), B, H, m, dk, dv,
                                        _dtype_code(q), _phi_code(phi), _stream(q.device)), "la_decode_verify")
    return out


def decode_commit(k: torch.Tensor, v: torch.Tensor, S: torch.Tensor, accepted: torch.Tensor, *,
                  phi: str = "identity") -> None:
    """S <- S + sum_{t < accepted[b]} k_t (x) v_t in place (the accepted drafts).

    k, v: [B, H, m, d]; S: fp32 [B, H, d, d]; accepted: int32 [B] on the device.
    """
    _need(k, "k", k.dtype, k.device)
    _need(v, "v", k.dtype, k.device)
    _need(S, "S", torch.float32, k.device)
    _need(accepted, "accepted", torch.int32, k.device)
    B, H, m, dk = k.shape
    dv = v.shape[-1]
    if tuple(S.shape) != (B, H, dk, dv) or accepted.numel() != B:
        raise ValueError("S must be [B, H, dk, dv] and accepted [B]")
    with torch.cuda.device(k.device):
        _abi.check(lib.la_decode_commit(_ptr(k), _ptr(v), _ptr(S), _ptr(accepted), B, H, m, dk, dv,
                                        _dtype_code(k), _phi_code(phi), _stream(k.device)), "la_decode_commit")


def _heads_view(t: torch.Tensor, name: str, dtype, device):
    """la_view of heads [B, H, N, d] or packed [T, H, d] (one batch entry), last dim contiguous."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    st, shape = t.stride(), t.shape
    if st[-1] != 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # the stride of a dimension of one entry (or none) says nothing
    if len(st) == 4:
        return _abi.View(t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0,
                         st[2] if shape[2] > 1 else 0)
    return _abi.View(t.data_ptr(), 0, st[1] if shape[1] > 1 else 0, st[0] if shape[0] > 1 else 0)


def _norm_rope_args(q, k, q_weight, k_weight, inv_freq, positions):
    """Checks of the arguments that both directions share; returns (B, N, Hq, Hk, d, positions' pointer, their
    width, strides, the weights' dtype code)."""
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if q.dim() not in (3, 4) or k.dim() != q.dim() or k.shape[-1] != q.shape[-1]:
        raise ValueError("q and k must be [B, H, N, d], or packed [T, H, d]")
    if q.dim() == 4:
        B, Hq, N, d = q.shape
        Hk, same = k.shape[1], k.shape[0] == B and k.shape[2] == N
    else:
        N, Hq, d = q.shape
        B, Hk, same = 1, k.shape[1], k.shape[0] == N
    if not same:
        raise ValueError("q and k must have the same tokens")
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        _need(t, n, None, q.device)
        if tuple(t.shape) != (d,):
            raise ValueError(f"{n} must be [d] = [{d}], got {tuple(t.shape)}")
    if q_weight.dtype != k_weight.dtype or q_weight.dtype not in (torch.float32, q.dtype):
        raise TypeError("q_weight and k_weight must both be float32, or both of q's dtype")
    rot = 0
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, q.device)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [rot / 2]")
        rot = 2 * inv_freq.numel()
    pos64, psb, psn = 0, 0, 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        if positions.device != q.device:
            raise ValueError(f"positions is on {positions.device}, expected {q.device}")
        pos64 = int(positions.dtype == torch.int64)
        if q.dim() == 4 and tuple(positions.shape) == (B, N):
            psb, psn = positions.stride()
        elif tuple(positions.shape) == (N,):
            psn = positions.stride(0)
        else:
            raise ValueError("positions must be [B, N] or [N] for [B, H, N, d], [T] for [T, H, d]")
    elif q.dim() == 3 and rot:
        raise ValueError("packed q and k need positions")
    return B, N, Hq, Hk, d, rot, pos64, psb, psn, _DT[q_weight.dtype]


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                 inv_freq: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, *,
                 eps: float = 1e-6, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Norm of every query and key head and rotation by the token's position.

    Each row x of d values becomes R(p) (w * x / sqrt(mean(x^2) + eps)): R turns
    the pairs (i, i + rot/2) -- (2i, 2i + 1) if interleaved -- of the first
    rot = 2 len(inv_freq) dims by the angle p * inv_freq[i] (norm only if
    inv_freq is None).  q [B, Hq, N, d] and k [B, Hk, N, d], or packed [T, H, d]
    (also one decode token of each sequence), of any strides with a contiguous
    last dim, e.g. slices of one projection's output; weights [d] in fp32 or q's
    dtype; inv_freq fp32; positions int32 / int64 [B, N] or [N] (default
    0 .. N-1), [T] for packed.  Returns contiguous (q_out, k_out), or writes the
    given ones (any strides).
    """
    dt = _dtype_code(q)
    B, N, Hq, Hk, d, rot, pos64, psb, psn, wdt = _norm_rope_args(q, k, q_weight, k_weight, inv_freq, positions)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
    k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device) if k_out is None else k_out
    if q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("q_out and k_out must have the shapes of q and k")
    views = [_heads_view(t, n, q.dtype, q.device)
             for t, n in ((q, "q"), (k, "k"), (q_out, "q_out"), (k_out, "k_out"))]
    with _on(q.device):
        _abi.check(lib.la_qk_norm_rope(*views, _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq), _ptr(positions), pos64,
                                       psb, psn, B, N, Hq, Hk, d, rot, eps, int(interleaved), dt, wdt,
                                       _stream(q.device)), "la_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          q_weight: torch.Tensor, k_weight: torch.Tensor, inv_freq: Optional[torch.Tensor] = None,
                          positions: Optional[torch.Tensor] = None, *, eps: float = 1e-6, interleaved: bool = False,
                          dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None):
    """Gradients of ``qk_norm_rope`` for dL/dq_out and dL/dk_out.

    q, k, weights, inv_freq, positions, eps and interleaved as in the forward
    call.  Returns (dq, dk, dq_weight, dk_weight): dq and dk in q's dtype
    (contiguous, or the given ones of any strides), the weight gradients fp32.
    """
    dt = _dtype_code(q)
    B, N, Hq, Hk, d, rot, pos64, psb, psn, wdt = _norm_rope_args(q, k, q_weight, k_weight, inv_freq, positions)
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device) if dq is None else dq
    dk = torch.empty(k.shape, dtype=q.dtype, device=q.device) if dk is None else dk
    for t, x, n in ((dq_out, q, "dq_out"), (dk_out, k, "dk_out"), (dq, q, "dq"), (dk, k, "dk")):
        if t.shape != x.shape:
            raise ValueError(f"{n} must be {tuple(x.shape)}, got {tuple(t.shape)}")
    views = [_heads_view(t, n, q.dtype, q.device) for t, n in
             ((dq_out, "dq_out"), (dk_out, "dk_out"), (q, "q"), (k, "k"), (dq, "dq"), (dk, "dk"))]
    dqw, dkw = (torch.empty(d, dtype=torch.float32, device=q.device) for _ in range(2))
    with _on(q.device):
        need = int(lib.la_qk_norm_rope_backward_workspace_size(d))
        workspace, ws_bytes = _workspace(workspace, need, q.device)
        _abi.check(lib.la_qk_norm_rope_backward(*views[:4], _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq),
                                                _ptr(positions), pos64, psb, psn, *views[4:], _ptr(dqw), _ptr(dkw), B,
                                                N, Hq, Hk, d, rot, eps, int(interleaved), dt, wdt, _ptr(workspace),
                                                ws_bytes, _stream(q.device)), "la_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


def device_status(clear: bool = True) -> int:
    """Device status word (0 = ok, 4 = a bounded device wait timed out). Synchronizes."""
    import ctypes
    v = ctypes.c_int(0)
    _abi.check(lib.la_device_status(ctypes.byref(v), 1 if clear else 0), "la_device_status")
    return int(v.value)
