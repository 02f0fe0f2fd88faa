"""Torch-facing wrappers of the C ABI (argument marshalling only).

Every step of the scan runs in the HIP kernels of libgdn.so; this module only
checks tensor placement, allocates outputs and workspace with torch, and passes
raw device pointers plus torch's current HIP stream across the ABI.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import GdnDesc, GdnError


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor (got %s)" % (name, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def make_desc(B, H, F, N, D, dtype: torch.dtype, *, gates_are_logits=False, eps=1e-6,
              normalize_keys=True, reverse=False) -> GdnDesc:
    if dtype == torch.bfloat16:
        io = _lib.GDN_BF16
    elif dtype == torch.float32:
        io = _lib.GDN_F32
    elif dtype == torch.float8_e4m3fn:
        io = _lib.GDN_FP8_E4M3
    else:
        raise TypeError("q/k/v must be bfloat16, float32 or float8_e4m3fn")
    flags = _lib.GDN_FLAG_GATES_ARE_LOGITS if gates_are_logits else 0
    if not normalize_keys:
        flags |= _lib.GDN_FLAG_NO_KEY_NORM
    if reverse:
        flags |= _lib.GDN_FLAG_REVERSE
    return GdnDesc(B, H, F, N, D, D, io, flags, float(eps))


def workspace_size(desc: GdnDesc) -> int:
    return int(_lib.load().gdn_workspace_size(ctypes.byref(desc)))


def alloc_workspace(desc: GdnDesc, device) -> Optional[torch.Tensor]:
    n = workspace_size(desc)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def _check_workspace(workspace, device):
    if workspace is None:
        return
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device:
        raise ValueError("workspace must be on %s (got %s)" % (device, workspace.device))
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")


def _run(fn_name, q, k, v, beta, alpha, S_in, o, S_out, workspace, desc, stream):
    lib = _lib.load()
    ws_bytes = 0 if workspace is None else workspace.numel()
    st = getattr(lib, fn_name)(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                               _ptr(alpha), _ptr(S_in), _ptr(o), _ptr(S_out), _ptr(workspace),
                               ctypes.c_size_t(ws_bytes), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, fn_name)


def _launch_stream(stream, device):
    return torch.cuda.current_stream(device) if stream is None else stream


def frame_scan_fwd(q, k, v, beta, alpha, S0=None, *, gates_are_logits: bool = False,
                   eps: float = 1e-6, normalize_keys: bool = True, reverse: bool = False,
                   o=None, S_final=None, workspace=None,
                   return_state: bool = True, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Whole-clip frame-wise GDN scan.

    q, k: [B,F,N,H,D]; v: [B,F,N,H,D] (bf16 or fp32, all the same dtype);
    beta: [B,F,N,H] fp32; alpha: [B,F,H] fp32; S0: [B,H,D,D] fp32 or None.
    reverse=True runs the recurrence from the last frame to the first.
    Returns (o [B,F,N,H,D] in the q dtype, S_final [B,H,D,D] fp32 or None).
    """
    B, F, N, H, D = q.shape
    _check(q, "q", q.dtype, (B, F, N, H, D))
    _check(k, "k", q.dtype, (B, F, N, H, D))
    _check(v, "v", q.dtype, (B, F, N, H, D))
    _check(beta, "beta", torch.float32, (B, F, N, H))
    _check(alpha, "alpha", torch.float32, (B, F, H))
    if S0 is not None:
        _check(S0, "S0", torch.float32, (B, H, D, D))
    desc = make_desc(B, H, F, N, D, q.dtype, gates_are_logits=gates_are_logits, eps=eps,
                     normalize_keys=normalize_keys, reverse=reverse)
    if o is not None:
        _check(o, "o", q.dtype, (B, F, N, H, D))
    if S_final is not None:
        _check(S_final, "S_final", torch.float32, (B, H, D, D))
    _check_workspace(workspace, q.device)
    stream = _launch_stream(stream, q.device)
    # Buffers allocated here belong to the launch stream, so torch's caching
    # allocator never hands them to other work while the kernels still run.
    with torch.cuda.stream(stream):
        if o is None:
            o = torch.empty_like(q)
        if S_final is None and return_state:
            S_final = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = alloc_workspace(desc, q.device)
        _run("gdn_frame_scan_fwd", q, k, v, beta, alpha, S0, o, S_final, workspace, desc, stream)
    return o, S_final


def frame_scan_fwd_static(q, k, v, beta, alpha, S0=None, *, gates_are_logits: bool = False,
                          eps: float = 1e-6, normalize_keys: bool = True, reverse: bool = False,
                          o=None, S_final=None,
                          return_state: bool = True, stream=None):
    """frame_scan_fwd through gdn_frame_scan_fwd_static: the library's own static
    scratch instead of a workspace.  The C entry point allocates nothing; pass
    o and S_final to keep this wrapper from allocating them with torch."""
    B, F, N, H, D = q.shape
    _check(q, "q", q.dtype, (B, F, N, H, D))
    _check(k, "k", q.dtype, (B, F, N, H, D))
    _check(v, "v", q.dtype, (B, F, N, H, D))
    _check(beta, "beta", torch.float32, (B, F, N, H))
    _check(alpha, "alpha", torch.float32, (B, F, H))
    if S0 is not None:
        _check(S0, "S0", torch.float32, (B, H, D, D))
    if o is not None:
        _check(o, "o", q.dtype, (B, F, N, H, D))
    if S_final is not None:
        _check(S_final, "S_final", torch.float32, (B, H, D, D))
    desc = make_desc(B, H, F, N, D, q.dtype, gates_are_logits=gates_are_logits, eps=eps,
                     normalize_keys=normalize_keys, reverse=reverse)
    stream = _launch_stream(stream, q.device)
    with torch.cuda.stream(stream):
        if o is None:
            o = torch.empty_like(q)
        if S_final is None and return_state:
            S_final = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device)
        st = _lib.load().gdn_frame_scan_fwd_static(
            ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S0),
            _ptr(o), _ptr(S_final), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, "gdn_frame_scan_fwd_static")
    return o, S_final


def frame_scan_fwd_fp8(q, q_scale, k, k_scale, v, v_scale, beta, alpha, S0=None, *,
                       gates_are_logits: bool = False, eps: float = 1e-6, normalize_keys: bool = True,
                       reverse: bool = False, o=None, S_final=None, workspace=None,
                       return_state: bool = True, stream=None):
    """frame_scan_fwd on block-scaled FP8 inputs (OCP MXFP8, E4M3 elements).

    q, k, v: [B,F,N,H,D] torch.float8_e4m3fn; q_scale, k_scale, v_scale:
    [B,F,N,H,D/32] torch.uint8 E8M0 exponents (value = e4m3 * 2^(s - 127));
    D in {32, 64, 128}.  Returns (o [B,F,N,H,D] bfloat16, S_final fp32 or None).
    """
    B, F, N, H, D = q.shape
    f8 = torch.float8_e4m3fn
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, f8, (B, F, N, H, D))
    nb = D // 32
    for name, t in (("q_scale", q_scale), ("k_scale", k_scale), ("v_scale", v_scale)):
        _check(t, name, torch.uint8, (B, F, N, H, nb))
    _check(beta, "beta", torch.float32, (B, F, N, H))
    _check(alpha, "alpha", torch.float32, (B, F, H))
    if S0 is not None:
        _check(S0, "S0", torch.float32, (B, H, D, D))
    if o is not None:
        _check(o, "o", torch.bfloat16, (B, F, N, H, D))
    if S_final is not None:
        _check(S_final, "S_final", torch.float32, (B, H, D, D))
    _check_workspace(workspace, q.device)
    desc = make_desc(B, H, F, N, D, f8, gates_are_logits=gates_are_logits, eps=eps,
                     normalize_keys=normalize_keys, reverse=reverse)
    stream = _launch_stream(stream, q.device)
    with torch.cuda.stream(stream):   # allocations belong to the launch stream
        if o is None:
            o = torch.empty((B, F, N, H, D), dtype=torch.bfloat16, device=q.device)
        if S_final is None and return_state:
            S_final = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = alloc_workspace(desc, q.device)
        ws_bytes = 0 if workspace is None else workspace.numel()
        st = _lib.load().gdn_frame_scan_fwd_fp8(
            ctypes.byref(desc), _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(v), _ptr(v_scale),
            _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(o), _ptr(S_final), _ptr(workspace),
            ctypes.c_size_t(ws_bytes), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, "gdn_frame_scan_fwd_fp8")
    return o, S_final


def frame_scan_fwd_fp4(q, q_scale, k, k_scale, v, v_scale, beta, alpha, S0=None, *,
                       gates_are_logits: bool = False, eps: float = 1e-6, normalize_keys: bool = True,
                       reverse: bool = False, o=None, S_final=None, workspace=None,
                       return_state: bool = True, stream=None):
    """frame_scan_fwd on block-scaled FP4 inputs (OCP MXFP4, E2M1 elements).

    q, k, v: [B,F,N,H,D/2] torch.uint8, two E2M1 codes per byte (feature 2j
    in the lower four bits of byte j); q_scale, k_scale, v_scale:
    [B,F,N,H,D/32] torch.uint8 E8M0 exponents; D in {32, 64, 128}.  Returns
    (o [B,F,N,H,D] bfloat16, S_final fp32 or None).
    """
    B, F, N, H, D2 = q.shape
    D = 2 * D2
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, torch.uint8, (B, F, N, H, D2))
    nb = D // 32
    for name, t in (("q_scale", q_scale), ("k_scale", k_scale), ("v_scale", v_scale)):
        _check(t, name, torch.uint8, (B, F, N, H, nb))
    _check(beta, "beta", torch.float32, (B, F, N, H))
    _check(alpha, "alpha", torch.float32, (B, F, H))
    if S0 is not None:
        _check(S0, "S0", torch.float32, (B, H, D, D))
    if o is not None:
        _check(o, "o", torch.bfloat16, (B, F, N, H, D))
    if S_final is not None:
        _check(S_final, "S_final", torch.float32, (B, H, D, D))
    _check_workspace(workspace, q.device)
    desc = make_desc(B, H, F, N, D, torch.bfloat16, gates_are_logits=gates_are_logits, eps=eps,
                     normalize_keys=normalize_keys, reverse=reverse)
    desc.io_dtype = _lib.GDN_FP4_E2M1
    stream = _launch_stream(stream, q.device)
    with torch.cuda.stream(stream):   # allocations belong to the launch stream
        if o is None:
            o = torch.empty((B, F, N, H, D), dtype=torch.bfloat16, device=q.device)
        if S_final is None and return_state:
            S_final = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = alloc_workspace(desc, q.device)
        ws_bytes = 0 if workspace is None else workspace.numel()
        st = _lib.load().gdn_frame_scan_fwd_fp4(
            ctypes.byref(desc), _ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(v), _ptr(v_scale),
            _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(o), _ptr(S_final), _ptr(workspace),
            ctypes.c_size_t(ws_bytes), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, "gdn_frame_scan_fwd_fp4")
    return o, S_final


def frame_step(q, k, v, beta, alpha, S_in=None, *, gates_are_logits: bool = False,
               eps: float = 1e-6, normalize_keys: bool = True, o=None, S_out=None, workspace=None, stream=None):
    """One frame of the scan for streaming use.

    q, k, v: [B,N,H,D] (or [B,1,N,H,D]); beta: [B,N,H] (or [B,1,N,H]);
    alpha: [B,H] (or [B,1,H]); S_in: [B,H,D,D] fp32 or None (zeros).
    S_out may be S_in itself (in-place carry).  Returns (o, S_out).
    """
    squeeze = q.dim() == 4
    if squeeze:
        q, k, v = q.unsqueeze(1), k.unsqueeze(1), v.unsqueeze(1)
        beta, alpha = beta.unsqueeze(1), alpha.unsqueeze(1)
        if o is not None:
            o = o.unsqueeze(1)
    B, F, N, H, D = q.shape
    if F != 1:
        raise ValueError("frame_step takes exactly one frame")
    _check(q, "q", q.dtype, (B, 1, N, H, D))
    _check(k, "k", q.dtype, (B, 1, N, H, D))
    _check(v, "v", q.dtype, (B, 1, N, H, D))
    _check(beta, "beta", torch.float32, (B, 1, N, H))
    _check(alpha, "alpha", torch.float32, (B, 1, H))
    if S_in is not None:
        _check(S_in, "S_in", torch.float32, (B, H, D, D))
    if o is not None:
        _check(o, "o", q.dtype, (B, 1, N, H, D))
    if S_out is not None:
        _check(S_out, "S_out", torch.float32, (B, H, D, D))
    _check_workspace(workspace, q.device)
    desc = make_desc(B, H, 1, N, D, q.dtype, gates_are_logits=gates_are_logits, eps=eps,
                     normalize_keys=normalize_keys)
    stream = _launch_stream(stream, q.device)
    with torch.cuda.stream(stream):   # allocations belong to the launch stream
        if o is None:
            o = torch.empty_like(q)
        if S_out is None:
            S_out = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = alloc_workspace(desc, q.device)
        _run("gdn_frame_step", q, k, v, beta, alpha, S_in, o, S_out, workspace, desc, stream)
    return (o.squeeze(1) if squeeze else o), S_out


def workspace_size_bwd(desc: GdnDesc) -> int:
    return int(_lib.load().gdn_workspace_size_bwd(ctypes.byref(desc)))


def saved_size(desc: GdnDesc) -> int:
    return int(_lib.load().gdn_saved_size(ctypes.byref(desc)))


def workspace_size_bwd_saved(desc: GdnDesc) -> int:
    return int(_lib.load().gdn_workspace_size_bwd_saved(ctypes.byref(desc)))


def frame_scan_fwd_save(q, k, v, beta, alpha, S0=None, *, gates_are_logits: bool = False,
                        eps: float = 1e-6, normalize_keys: bool = True, reverse: bool = False,
                        o=None, S_final=None, saved=None, return_state: bool = True, stream=None):
    """frame_scan_fwd that also keeps, in `saved` (a uint8 device tensor of
    gdn_saved_size bytes, allocated when None), what frame_scan_bwd(...,
    saved=saved) reads instead of recomputing.  Returns (o, S_final, saved)."""
    B, F, N, H, D = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, q.dtype, (B, F, N, H, D))
    _check(beta, "beta", torch.float32, (B, F, N, H))
    _check(alpha, "alpha", torch.float32, (B, F, H))
    if S0 is not None:
        _check(S0, "S0", torch.float32, (B, H, D, D))
    if o is not None:
        _check(o, "o", q.dtype, (B, F, N, H, D))
    if S_final is not None:
        _check(S_final, "S_final", torch.float32, (B, H, D, D))
    _check_workspace(saved, q.device)
    desc = make_desc(B, H, F, N, D, q.dtype, gates_are_logits=gates_are_logits, eps=eps,
                     normalize_keys=normalize_keys, reverse=reverse)
    stream = _launch_stream(stream, q.device)
    with torch.cuda.stream(stream):   # allocations belong to the launch stream
        if o is None:
            o = torch.empty_like(q)
        if S_final is None and return_state:
            S_final = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device)
        if saved is None:
            saved = torch.empty(max(saved_size(desc), 1), dtype=torch.uint8, device=q.device)
        st = _lib.load().gdn_frame_scan_fwd_save(
            ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(o),
            _ptr(S_final), _ptr(saved), ctypes.c_size_t(saved.numel()), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, "gdn_frame_scan_fwd_save")
    return o, S_final, saved


def frame_scan_bwd(q, k, v, beta, alpha, dO, S0=None, dS_final=None, *, gates_are_logits: bool = False,
                   eps: float = 1e-6, normalize_keys: bool = True, reverse: bool = False,
                   workspace=None, return_dS0: bool = True, saved=None, stream=None):
    """Gradients of frame_scan_fwd with respect to its inputs.

    q, k, v, beta, alpha, S0 and the flags as for frame_scan_fwd; dO: [B,F,N,H,D]
    in the q dtype (the loss gradient of o); dS_final: [B,H,D,D] fp32 or None
    (zeros).  Returns (dq, dk, dv, dbeta, dalpha, dS0): dq, dk, dv in the q
    dtype, the rest fp32 (dbeta and dalpha are logit gradients with
    gates_are_logits; dS0 is None when return_dS0 is False).  With `saved`
    (from frame_scan_fwd_save on the same inputs) the per-frame operands of
    the forward walk are read from it instead of recomputed, and S0 is unused.
    """
    B, F, N, H, D = q.shape
    _check(q, "q", q.dtype, (B, F, N, H, D))
    _check(k, "k", q.dtype, (B, F, N, H, D))
    _check(v, "v", q.dtype, (B, F, N, H, D))
    _check(beta, "beta", torch.float32, (B, F, N, H))
    _check(alpha, "alpha", torch.float32, (B, F, H))
    _check(dO, "dO", q.dtype, (B, F, N, H, D))
    if S0 is not None:
        _check(S0, "S0", torch.float32, (B, H, D, D))
    if dS_final is not None:
        _check(dS_final, "dS_final", torch.float32, (B, H, D, D))
    _check_workspace(workspace, q.device)
    desc = make_desc(B, H, F, N, D, q.dtype, gates_are_logits=gates_are_logits, eps=eps,
                     normalize_keys=normalize_keys, reverse=reverse)
    stream = _launch_stream(stream, q.device)
    with torch.cuda.stream(stream):   # allocations belong to the launch stream
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dbeta, dalpha = torch.empty_like(beta), torch.empty_like(alpha)
        dS0 = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device) if return_dS0 else None
        lib = _lib.load()
        if workspace is None:
            n = workspace_size_bwd_saved(desc) if saved is not None else workspace_size_bwd(desc)
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n > 0 else None
        ws_bytes = 0 if workspace is None else workspace.numel()
        if saved is not None:
            name = "gdn_frame_scan_bwd_saved"
            st = lib.gdn_frame_scan_bwd_saved(
                ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(dO),
                _ptr(dS_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dalpha), _ptr(dS0),
                _ptr(saved), ctypes.c_size_t(saved.numel()), _ptr(workspace), ctypes.c_size_t(ws_bytes),
                ctypes.c_void_p(stream.cuda_stream))
        else:
            name = "gdn_frame_scan_bwd"
            st = lib.gdn_frame_scan_bwd(
                ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(S0), _ptr(dO),
                _ptr(dS_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dalpha), _ptr(dS0),
                _ptr(workspace), ctypes.c_size_t(ws_bytes), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, name)
    return dq, dk, dv, dbeta, dalpha, dS0


def profile_begin() -> None:
    st = _lib.load().gdn_profile_begin()
    if st != 0:
        raise GdnError(st, "gdn_profile_begin")


def profile_end() -> dict:
    """Stop profiling; {kernel name: (total ms, launches)} for every kernel kind."""
    lib = _lib.load()
    ms = (ctypes.c_double * _lib.GDN_NUM_KERNELS)()
    n = (ctypes.c_int64 * _lib.GDN_NUM_KERNELS)()
    st = lib.gdn_profile_end(ms, n)
    if st != 0:
        raise GdnError(st, "gdn_profile_end")
    return {lib.gdn_kernel_name(i).decode(): (ms[i], int(n[i])) for i in range(_lib.GDN_NUM_KERNELS)}


def block_workspace_size(B, H, F, N, D, C) -> int:
    desc = make_desc(B, H, F, N, D, torch.bfloat16)
    return int(_lib.load().gdn_block_workspace_size(ctypes.byref(desc), int(C)))


def block_in_proj(x, w_qkv, w_gate, *, H: int, D: int, q=None, k=None, v=None, beta_logit=None,
                  alpha_logit=None, workspace=None, stream=None):
    """Input projections of a GDN block: hidden states to the scan's inputs.

    x: [B,F,N,C] bf16; w_qkv: [3,H,D,C] bf16; w_gate: [2,H,C] bf16 (weights
    output-major, as torch.nn.Linear stores them).  Returns
    (q, k, v, beta_logit, alpha_logit): q, k, v [B,F,N,H,D] bf16,
    beta_logit [B,F,N,H] fp32 (one per token) and alpha_logit [B,F,H] fp32
    (the frame mean of the per-token alpha terms); the logits feed
    frame_scan_fwd(..., gates_are_logits=True).
    """
    B, F, N, C = x.shape
    _check(x, "x", torch.bfloat16, (B, F, N, C))
    _check(w_qkv, "w_qkv", torch.bfloat16, (3, H, D, C))
    _check(w_gate, "w_gate", torch.bfloat16, (2, H, C))
    outs = {"q": q, "k": k, "v": v}
    for name, t in outs.items():
        if t is not None:
            _check(t, name, torch.bfloat16, (B, F, N, H, D))
    if beta_logit is not None:
        _check(beta_logit, "beta_logit", torch.float32, (B, F, N, H))
    if alpha_logit is not None:
        _check(alpha_logit, "alpha_logit", torch.float32, (B, F, H))
    _check_workspace(workspace, x.device)
    desc = make_desc(B, H, F, N, D, torch.bfloat16)
    lib = _lib.load()
    stream = _launch_stream(stream, x.device)
    with torch.cuda.stream(stream):   # allocations belong to the launch stream
        q, k, v = [t if t is not None else torch.empty((B, F, N, H, D), dtype=torch.bfloat16, device=x.device)
                   for t in (q, k, v)]
        if beta_logit is None:
            beta_logit = torch.empty((B, F, N, H), dtype=torch.float32, device=x.device)
        if alpha_logit is None:
            alpha_logit = torch.empty((B, F, H), dtype=torch.float32, device=x.device)
        if workspace is None:
            n = int(lib.gdn_block_workspace_size(ctypes.byref(desc), int(C)))
            workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
        st = lib.gdn_block_in_proj(ctypes.byref(desc), int(C), _ptr(x), _ptr(w_qkv), _ptr(w_gate), _ptr(q),
                                   _ptr(k), _ptr(v), _ptr(beta_logit), _ptr(alpha_logit), _ptr(workspace),
                                   ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, "gdn_block_in_proj")
    return q, k, v, beta_logit, alpha_logit


def block_out_proj(o, w_out, *, y=None, workspace=None, stream=None):
    """Output projection of a GDN block: y [B,F,N,C] bf16 = o [B,F,N,H,D] bf16
    (flattened to H*D) times the transpose of w_out [C, H*D] bf16."""
    B, F, N, H, D = o.shape
    C = w_out.shape[0]
    _check(o, "o", torch.bfloat16, (B, F, N, H, D))
    _check(w_out, "w_out", torch.bfloat16, (C, H * D))
    if y is not None:
        _check(y, "y", torch.bfloat16, (B, F, N, C))
    _check_workspace(workspace, o.device)
    desc = make_desc(B, H, F, N, D, torch.bfloat16)
    lib = _lib.load()
    stream = _launch_stream(stream, o.device)
    with torch.cuda.stream(stream):
        if y is None:
            y = torch.empty((B, F, N, C), dtype=torch.bfloat16, device=o.device)
        if workspace is None:
            n = int(lib.gdn_block_workspace_size(ctypes.byref(desc), int(C)))
            workspace = torch.empty(n, dtype=torch.uint8, device=o.device)
        st = lib.gdn_block_out_proj(ctypes.byref(desc), int(C), _ptr(o), _ptr(w_out), _ptr(y), _ptr(workspace),
                                    ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(stream.cuda_stream))
    if st != 0:
        raise GdnError(st, "gdn_block_out_proj")
    return y


def _io(dtype: torch.dtype, what: str) -> int:
    if dtype == torch.bfloat16:
        return _lib.GDN_BF16
    if dtype == torch.float32:
        return _lib.GDN_F32
    raise TypeError("%s must be bfloat16 or float32 (got %s)" % (what, dtype))


def _same_device(x, **tensors):
    index = x.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError("%s must be on %s (got %s)" % (name, x.device, t.device))


_HERE = contextlib.nullcontext()
# the tensors at hand have initialised the device layer, so its own check of that is left out
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# the current stream's handle without a Stream object around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(stream, device):
    """(context, stream handle) of a launch: what is allocated within the context
    belongs to the stream.  The current stream of the current device, the usual
    case, needs no context (entering one costs as much as a small kernel)."""
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream must be on %s (got %s)" % (device, stream.device))
        return torch.cuda.stream(stream), stream.cuda_stream
    index = device.index
    return (_HERE if index == _current_device() else torch.cuda.device(device)), _raw_stream(index)


def _workspace(workspace, n: int, device):
    """The caller's workspace, or one of n bytes from the current stream's allocator."""
    if workspace is not None or n == 0:
        return workspace
    return torch.empty(n, dtype=torch.uint8, device=device)


def _ws_bytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel()


def _norm_desc(x, weight, bias, eps):
    C = x.shape[-1] if x.dim() else 0
    rows = x.numel() // C if C else 0
    w_dtype = torch.float32 if weight is None and bias is None else (bias if weight is None else weight).dtype
    if weight is not None:
        _check(weight, "weight", w_dtype, (C,))
    if bias is not None:
        _check(bias, "bias", w_dtype, (C,))
    return _lib.GdnNormDesc(rows, C, _io(x.dtype, "x"), _io(w_dtype, "weight"), eps)


def layer_norm_fwd(x, weight=None, bias=None, *, eps: float = 1e-6, y=None, mean=None, rstd=None,
                   return_stats: bool = True, stream=None):
    """Layer norm over the last axis: y = (x - mean) * rstd * weight + bias.

    x: [..., C] bf16 or fp32; weight, bias: [C] in x's dtype or fp32 (both the
    same), or None.  Returns (y, mean, rstd): y like x, mean and rstd [...]
    fp32, which layer_norm_bwd reads (None with return_stats=False unless
    passed in).
    """
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    _check(x, "x", x.dtype, x.shape)
    desc = _norm_desc(x, weight, bias, eps)
    stats = x.shape[:-1]
    if y is not None:
        _check(y, "y", x.dtype, x.shape)
    if mean is not None:
        _check(mean, "mean", torch.float32, stats)
    if rstd is not None:
        _check(rstd, "rstd", torch.float32, stats)
    _same_device(x, weight=weight, bias=bias, y=y, mean=mean, rstd=rstd)
    where, handle = _launch(stream, x.device)
    with where:   # allocations belong to the launch stream
        if y is None:
            y = torch.empty_like(x)
        if mean is None and return_stats:
            mean = torch.empty(stats, dtype=torch.float32, device=x.device)
        if rstd is None and return_stats:
            rstd = torch.empty(stats, dtype=torch.float32, device=x.device)
        st = _lib.load().gdn_layer_norm_fwd(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y),
                                            _ptr(mean), _ptr(rstd), handle)
    if st != 0:
        raise GdnError(st, "gdn_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, weight=None, bias=None, *, dx=None, dweight=None, dbias=None,
                   workspace=None, stream=None):
    """Gradients of layer_norm_fwd.

    dy: the loss gradient of y, like x; mean, rstd: the forward call's; weight
    and bias as given to it (bias only says that its gradient is wanted).
    Returns (dx, dweight, dbias): dx like x, the others in the weight's dtype,
    None where the parameter is None.
    """
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    _check(x, "x", x.dtype, x.shape)
    _check(dy, "dy", x.dtype, x.shape)
    desc = _norm_desc(x, weight, bias, 1.0)   # eps acts through rstd
    stats = x.shape[:-1]
    _check(mean, "mean", torch.float32, stats)
    _check(rstd, "rstd", torch.float32, stats)
    if dx is not None:
        _check(dx, "dx", x.dtype, x.shape)
    for name, t, p in (("dweight", dweight, weight), ("dbias", dbias, bias)):
        if t is not None:
            if p is None:
                raise ValueError("%s needs its parameter" % name)
            _check(t, name, p.dtype, p.shape)
    _check_workspace(workspace, x.device)
    _same_device(x, dy=dy, mean=mean, rstd=rstd, weight=weight, bias=bias, dx=dx, dweight=dweight, dbias=dbias)
    lib = _lib.load()
    where, handle = _launch(stream, x.device)
    with where:   # allocations belong to the launch stream
        if dx is None:
            dx = torch.empty_like(x)
        if dweight is None and weight is not None:
            dweight = torch.empty_like(weight)
        if dbias is None and bias is not None:
            dbias = torch.empty_like(bias)
        if weight is not None or bias is not None:
            workspace = _workspace(workspace, int(lib.gdn_layer_norm_workspace_size(ctypes.byref(desc))), x.device)
        st = lib.gdn_layer_norm_bwd(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd),
                                    _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(workspace), _ws_bytes(workspace),
                                    handle)
    if st != 0:
        raise GdnError(st, "gdn_layer_norm_bwd")
    return dx, dweight, dbias


def video_positions(F: int, Hg: int, Wg: int, *, frame_offset: int = 0, device="cuda") -> torch.Tensor:
    """Positions of a video clip's tokens for rotary(): int32 [F, Hg*Wg, 3]
    with (frame_offset + frame, row, column) of each token."""
    axes = [torch.arange(n, dtype=torch.int32, device=device) for n in (F, Hg, Wg)]
    axes[0] += frame_offset
    return torch.stack(torch.meshgrid(*axes, indexing="ij"), dim=-1).reshape(F, Hg * Wg, 3).contiguous()


def rotary(q, k, pos, *, axes, theta: float = 10000.0, halves: bool = False, inverse: bool = False, q_out=None,
           k_out=None, stream=None):
    """Rotary positions over several axes, for queries and keys in one launch.

    q: [..., Hq, D] and k: [..., Hk, D], bf16 or fp32, the same leading (token)
    shape; k (or q) may be None.  pos: int32 or float32 [..., A], its leading
    shape the last of q's token axes (a batch shares its positions).  axes: A
    even numbers, the features each axis turns; features past their sum pass
    through.  inverse=True turns back (also the gradient).  q_out and k_out may
    be q and k.  Returns (q_out, k_out).
    """
    x = q if q is not None else k
    if not isinstance(x, torch.Tensor):
        raise TypeError("q or k must be a torch.Tensor")
    if x.dim() < 2:
        raise ValueError("q and k must be [..., H, D]")
    lead, D = tuple(x.shape[:-2]), x.shape[-1]
    heads = {}
    for name, t, out in (("q", q, q_out), ("k", k, k_out)):
        if t is None:
            if out is not None:
                raise ValueError("%s_out without %s" % (name, name))
            heads[name] = 0
            continue
        if t.dim() != x.dim():
            raise ValueError("q and k must have the same token axes")
        _check(t, name, x.dtype, lead + (t.shape[-2], D))
        heads[name] = t.shape[-2]
        if out is not None:
            _check(out, name + "_out", t.dtype, t.shape)
    if not isinstance(pos, torch.Tensor) or pos.dtype not in (torch.int32, torch.float32):
        raise TypeError("pos must be an int32 or float32 tensor")
    axes = [int(d) for d in axes]
    if not 1 <= len(axes) <= _lib.GDN_ROTARY_MAX_AXES:
        raise ValueError("1 to %d axes are supported (got %d)" % (_lib.GDN_ROTARY_MAX_AXES, len(axes)))
    n = pos.dim() - 1
    if n < 0 or n > len(lead):
        raise ValueError("pos must be [..., %d] over q's last token axes" % len(axes))
    _check(pos, "pos", pos.dtype, lead[len(lead) - n:] + (len(axes),))
    _same_device(x, q=q, k=k, pos=pos, q_out=q_out, k_out=k_out)
    tokens = 1
    for s in lead:
        tokens *= s
    flags = ((_lib.GDN_FLAG_ROTARY_HALVES if halves else 0) | (_lib.GDN_FLAG_ROTARY_INVERSE if inverse else 0) |
             (_lib.GDN_FLAG_ROTARY_POS_F32 if pos.dtype == torch.float32 else 0))
    dims = (ctypes.c_int32 * _lib.GDN_ROTARY_MAX_AXES)(*axes)
    desc = _lib.GdnRotaryDesc(tokens, pos.numel() // len(axes), heads["q"], heads["k"], D, len(axes), dims,
                              _io(x.dtype, "q and k"), flags, float(theta))
    where, handle = _launch(stream, x.device)
    with where:   # allocations belong to the launch stream
        if q is not None and q_out is None:
            q_out = torch.empty_like(q)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k)
        st = _lib.load().gdn_rotary(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(pos), _ptr(q_out), _ptr(k_out),
                                    handle)
    if st != 0:
        raise GdnError(st, "gdn_rotary")
    return q_out, k_out


def _token_strides(t, name):
    """(token stride, tokens between sequences or 0 for packed) of t [..., H, D]:
    heads packed, a sequence's tokens evenly apart."""
    H, D = t.shape[-2:]
    if t.is_contiguous() or t.numel() == 0:
        return H * D, 0
    ok = (D == 1 or t.stride(-1) == 1) and (H == 1 or t.stride(-2) == D)
    axes = [i for i in range(t.dim() - 2) if t.shape[i] > 1]
    batch = bool(axes) and t.dim() > 3 and axes[0] == 0
    inner = axes[1:] if batch else axes
    # one token a sequence: the step between the sequences is the token stride
    ld = t.stride(inner[-1]) if inner else t.stride(0) if batch else H * D
    ok = ok and ld >= H * D                   # not broadcast (0 would mean packed), no tokens that overlap
    step = ld
    for i in reversed(inner):                 # the token axes continue one step
        ok = ok and t.stride(i) == step
        step *= t.shape[i]
    room = 0
    if ok and batch and inner and t.stride(0) != step:
        room = t.stride(0) // ld
        ok = t.stride(0) % ld == 0 and t.stride(0) > step
    if not ok:
        raise ValueError("%s must have packed heads and evenly spaced tokens" % name)
    return ld, room


def _attn_args(q, k, v, causal, causal_block, scale, cu_q, cu_k, max_q, max_k):
    """Checks shared by attention_fwd and attention_bwd: (desc, cu_q, cu_k)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
    sq, sk = q.shape, k.shape
    dims = len(sq)
    if not 3 <= dims <= 5 or len(sk) != dims or v.shape != sk:
        raise ValueError("q, k and v must be [T, H, D], [B, L, H, D] or [B, F, N, H, D], k and v alike (got %s, %s, %s)"
                         % (tuple(sq), tuple(sk), tuple(v.shape)))
    Hq, D = sq[-2:]
    Hk = sk[-2]
    if sk[-1] != D:
        raise ValueError("q and k must have the same head size")
    io = _io(q.dtype, "q, k and v")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError("%s must be a device tensor (got %s)" % (name, t.device))
        if t.dtype != q.dtype:
            raise TypeError("%s must be %s (got %s)" % (name, q.dtype, t.dtype))
    if q.is_contiguous() and k.is_contiguous() and v.is_contiguous():
        ldq = ldk = ldv = rk = 0
    else:
        (ldq, rq), (ldk, rk), (ldv, rv) = [_token_strides(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v"))]
        if rq:
            raise ValueError("q must have packed heads and evenly spaced tokens")
        if rk != rv:
            raise ValueError("the sequences of k and v must lie equally far apart")
    if dims == 3:
        if cu_q is None:
            raise ValueError("packed q [T, H, D] needs cu_q")
        tq, tk = sq[0], sk[0]
        cu_k = cu_q if cu_k is None else cu_k
        n_seq = cu_q.numel() - 1
        if n_seq < 0:
            raise ValueError("cu_q must hold n_seq + 1 offsets")
        _check(cu_q, "cu_q", torch.int32, (n_seq + 1,))
        _check(cu_k, "cu_k", torch.int32, (n_seq + 1,))
        max_q = tq if max_q is None else min(int(max_q), tq)
        max_k = tk if max_k is None else min(int(max_k), tk)
    else:
        if cu_q is not None or cu_k is not None or max_q is not None or max_k is not None:
            raise ValueError("cu_q, cu_k, max_q and max_k belong to packed q [T, H, D]")
        n_seq = sq[0]
        if sk[0] != n_seq:
            raise ValueError("q and k must have the same batch size")
        max_q, max_k = sq[1:-2].numel(), sk[1:-2].numel()
        tq, tk = n_seq * max_q, n_seq * max_k
    if causal_block is None:
        causal_block = sq[2] if dims == 5 else 1
    _same_device(q, k=k, v=v, cu_q=cu_q, cu_k=cu_k)
    desc = _lib.GdnAttnDesc(tq, tk, ldq, ldk, ldv, rk, n_seq, Hq, Hk, D, max_q, max_k,
                            min(int(causal_block), 2 ** 31 - 1), io,
                            _lib.GDN_FLAG_ATTN_CAUSAL if causal else 0, D ** -0.5 if scale is None else scale)
    return desc, cu_q, cu_k


def _like(t):
    """An uninitialised contiguous tensor like t."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def attention_fwd(q, k, v, *, causal: bool = False, causal_block: Optional[int] = None, scale=None, cu_q=None,
                  cu_k=None, max_q=None, max_k=None, k_len=None, o=None, lse=None, return_lse: bool = True,
                  workspace=None, stream=None):
    """Softmax attention with grouped heads.

    q: [B, L, Hq, D], k and v: [B, Lk, Hk, D] (or [B, F, N, H, D] frames, or
    packed [T, H, D] with cu_q), bf16 or fp32, Hq a multiple of Hk, D in {16,
    32, 64, 128}; heads packed, tokens evenly apart (a slice of a fused
    projection, the first tokens k[:, :n] of a cache's slots, or single tokens
    q[:, -1:] of long sequences will do; broadcast views will not).
    causal=True: the queries are the last positions of
    their sequence and see the keys up to the end of their own block of
    causal_block positions (default: a frame's N tokens for [B, F, N, H, D],
    else 1).  cu_q, cu_k (default cu_q): int32 [n_seq + 1] offsets of packed
    sequences, max_q and max_k bounds of their lengths (default: all tokens;
    the tighter, the fewer empty workgroups).  k_len: int32 [n_seq], keys in use
    of each sequence's (a cache with room).  Returns (o like q, lse [..., Hq]
    fp32 or None); tokens of no sequence are left unset.
    """
    desc, cu_q, cu_k = _attn_args(q, k, v, causal, causal_block, scale, cu_q, cu_k, max_q, max_k)
    if k_len is not None:
        _check(k_len, "k_len", torch.int32, (desc.n_seq,))
    if o is not None:
        _check(o, "o", q.dtype, q.shape)
    if lse is not None:
        _check(lse, "lse", torch.float32, q.shape[:-1])
    _check_workspace(workspace, q.device)
    _same_device(q, k_len=k_len, o=o, lse=lse)
    lib = _lib.load()
    where, handle = _launch(stream, q.device)
    with where:   # allocations belong to the launch stream
        if o is None:
            o = _like(q)
        if lse is None and return_lse:
            lse = q.new_empty(q.shape[:-1], dtype=torch.float32)
        workspace = _workspace(workspace, int(lib.gdn_attn_workspace_size(ctypes.byref(desc))), q.device)
        st = lib.gdn_attn_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), _ptr(k_len),
                              _ptr(o), _ptr(lse), _ptr(workspace), _ws_bytes(workspace),
                              handle)
    if st != 0:
        raise GdnError(st, "gdn_attn_fwd")
    return o, lse


def attention_bwd(q, k, v, o, lse, dO, *, causal: bool = False, causal_block: Optional[int] = None, scale=None,
                  cu_q=None, cu_k=None, max_q=None, max_k=None, dq=None, dk=None, dv=None, workspace=None,
                  stream=None):
    """Gradients of attention_fwd (without k_len): (dq, dk, dv) in the inputs'
    dtype, contiguous.  o and lse are the forward call's, dO the loss gradient
    of o; the rest as given to it.  Tokens of no sequence are left unset."""
    desc, cu_q, cu_k = _attn_args(q, k, v, causal, causal_block, scale, cu_q, cu_k, max_q, max_k)
    _check(o, "o", q.dtype, q.shape)
    _check(lse, "lse", torch.float32, q.shape[:-1])
    _check(dO, "dO", q.dtype, q.shape)
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _check(t, name, like.dtype, like.shape)
    _check_workspace(workspace, q.device)
    _same_device(q, o=o, lse=lse, dO=dO, dq=dq, dk=dk, dv=dv)
    lib = _lib.load()
    where, handle = _launch(stream, q.device)
    with where:   # allocations belong to the launch stream
        dq = _like(q) if dq is None else dq
        dk = _like(k) if dk is None else dk
        dv = _like(v) if dv is None else dv
        workspace = _workspace(workspace, int(lib.gdn_attn_workspace_size_bwd(ctypes.byref(desc))), q.device)
        st = lib.gdn_attn_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(cu_q),
                              _ptr(cu_k), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), _ws_bytes(workspace),
                              handle)
    if st != 0:
        raise GdnError(st, "gdn_attn_bwd")
    return dq, dk, dv


# ------------------------------------------------------------------ 8-bit projections
FP8_GROUP = 128   # columns of an activation's scale, rows and columns of a weight's


def _fp8_out(x, y, y_scale):
    """Checks of the outputs of rms_norm_fwd_fp8 and quantize_fp8: the scales' shape."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() < 1:
        raise ValueError("x must be [..., C]")
    if not (x.is_cuda and x.is_contiguous()):
        _check(x, "x", x.dtype, x.shape)
    shape = x.shape
    scales = shape[:-1] + (-(-shape[-1] // FP8_GROUP),)
    if y is not None:
        _check(y, "y", torch.float8_e4m3fn, shape)
    if y_scale is not None:
        _check(y_scale, "y_scale", torch.float32, scales)
    return scales


def rms_norm_fwd_fp8(x, weight=None, residual=None, *, eps: float = 1e-6, y=None, y_scale=None, total=None,
                     stream=None):
    """Root-mean-square norm over the last axis with an 8-bit output, for the
    projections of matmul_fp8: y = t * (<t^2> + eps)^(-1/2) * weight, t = x + residual.

    x: [..., C] bf16 or fp32; weight: [C] in x's dtype or fp32, or None; residual:
    like x, or None.  Returns (y, y_scale, total): y float8_e4m3fn like x, y_scale
    [..., ceil(C / 128)] fp32, one for each group of 128 columns (a value is its code
    times its scale), and total = t in x's dtype (None without a residual), which may
    be given as x or residual itself.  Any C will do here; matmul_fp8 takes multiples of
    16.  Forward only, as all of this section: the outputs carry no gradient, whatever
    the inputs ask for.
    """
    scales = _fp8_out(x, y, y_scale)
    desc = _norm_desc(x, weight, None, eps)
    if residual is not None:
        _check(residual, "residual", x.dtype, x.shape)
    if total is not None:
        if residual is None:
            raise ValueError("total needs a residual")
        _check(total, "total", x.dtype, x.shape)
    _same_device(x, weight=weight, residual=residual, y=y, y_scale=y_scale, total=total)
    where, handle = _launch(stream, x.device)
    with where:   # allocations belong to the launch stream
        if y is None:
            y = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        if y_scale is None:
            y_scale = x.new_empty(scales, dtype=torch.float32)
        if total is None and residual is not None:
            total = torch.empty_like(x)
        st = _lib.load().gdn_rms_norm_fwd_fp8(ctypes.byref(desc), _ptr(x), _ptr(residual), _ptr(weight), _ptr(total),
                                              _ptr(y), _ptr(y_scale), handle)
    if st != 0:
        raise GdnError(st, "gdn_rms_norm_fwd_fp8")
    return y, y_scale, total


def quantize_fp8(x, *, y=None, y_scale=None, stream=None):
    """x [..., C] (bf16 or fp32) in 8 bits with a scale for each group of 128
    columns, as rms_norm_fwd_fp8 gives its output: (y, y_scale), without a gradient."""
    scales = _fp8_out(x, y, y_scale)
    desc = _norm_desc(x, None, None, 1.0)
    _same_device(x, y=y, y_scale=y_scale)
    where, handle = _launch(stream, x.device)
    with where:   # allocations belong to the launch stream
        if y is None:
            y = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        if y_scale is None:
            y_scale = x.new_empty(scales, dtype=torch.float32)
        st = _lib.load().gdn_quantize_fp8(ctypes.byref(desc), _ptr(x), _ptr(y), _ptr(y_scale), handle)
    if st != 0:
        raise GdnError(st, "gdn_quantize_fp8")
    return y, y_scale


def matmul_fp8(x, x_scale, w, w_scale, *, parts: int = 1, y=None, stream=None):
    """Product of 8-bit floats with fp32 scales: y = x w^T.

    x: [..., K] float8_e4m3fn with x_scale [..., ceil(K / 128)] fp32
    (rms_norm_fwd_fp8, quantize_fp8); w: [N, K] float8_e4m3fn, output-major, with
    w_scale [ceil(N / 128), ceil(K / 128)] fp32 (inputs.to_fp8_weight); K a multiple
    of 16.  Returns y [..., N] bf16, or with parts > 1 [parts, ..., N / parts].
    Forward only: y carries no gradient.
    """
    for name, t in (("x", x), ("w", w)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
    if x.dim() < 1 or w.dim() != 2:
        raise ValueError("x must be [..., K] and w [N, K]")
    N, K = w.shape
    lead = x.shape[:-1]
    parts = int(parts)
    if parts < 1 or N % parts:
        raise ValueError("parts must divide N = %d (got %d)" % (N, parts))
    _check(x, "x", torch.float8_e4m3fn, lead + (K,))
    _check(w, "w", torch.float8_e4m3fn, (N, K))
    kb = -(-K // FP8_GROUP)
    _check(x_scale, "x_scale", torch.float32, lead + (kb,))
    _check(w_scale, "w_scale", torch.float32, (-(-N // FP8_GROUP), kb))
    shape = lead + (N,) if parts == 1 else (parts,) + lead + (N // parts,)
    if y is not None:
        _check(y, "y", torch.bfloat16, shape)
    _same_device(x, x_scale=x_scale, w=w, w_scale=w_scale, y=y)
    desc = _lib.GdnMatmulDesc(lead.numel(), N, K, parts)
    where, handle = _launch(stream, x.device)
    with where:   # allocations belong to the launch stream
        if y is None:
            y = x.new_empty(shape, dtype=torch.bfloat16)
        st = _lib.load().gdn_matmul_fp8(ctypes.byref(desc), _ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(y),
                                        handle)
    if st != 0:
        raise GdnError(st, "gdn_matmul_fp8")
    return y


# ------------------------------------------------------------------ block-scaled caches
MX_BLOCK = 32     # features of a cache's scale


def cache_empty(*lead: int, H: int, D: int, fp4: bool, device="cuda"):
    """A cache of zeros for [*lead] tokens (slots and places, or packed tokens) of H
    heads of D features: (k, k_scale, v, v_scale), MXFP4 (uint8 [*lead, H, D/2]) or
    MXFP8 (float8_e4m3fn [*lead, H, D]) with E8M0 scales uint8 [*lead, H, D/32].  Slots
    of many requests are best not a power of two of bytes apart: 256 requests of 1000
    keys, 8 heads of 128 in MXFP4, are read in 100 us from slots of 33001 places and in
    220 from slots of 32768."""
    if D % MX_BLOCK:
        raise ValueError("D must be a multiple of %d (got %d)" % (MX_BLOCK, D))
    out = []
    for _ in range(2):
        codes = torch.zeros(lead + (H, D // 2 if fp4 else D), dtype=torch.uint8, device=device)
        out += [codes if fp4 else codes.view(torch.float8_e4m3fn),
                torch.zeros(lead + (H, D // MX_BLOCK), dtype=torch.uint8, device=device)]
    return tuple(out)


def _packed_tokens(t, name):
    """Places from one slot of t [..., H, X] to the next, 0: packed."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    ld, room = _token_strides(t, name)
    row = t.shape[-2] * t.shape[-1]
    # slots of one place, their step the token stride (packed [T, H, X] has no slots: its tokens must be packed)
    if ld != row and t.dim() > 3 and t.shape[1:-2].numel() == 1 and ld % row == 0:
        return ld // row
    if ld != row:
        raise ValueError("%s must have packed tokens" % name)
    return room


def _cache_args(k, k_scale, v, v_scale, fp4):
    """Checks of a cache: (places' shape, H, D, places between slots or 0)."""
    for name, t in (("k", k), ("k_scale", k_scale), ("v", v), ("v_scale", v_scale)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
    if not 3 <= k.dim() <= 5:
        raise ValueError("k must be [T, H, D], [B, L, H, D] or [B, F, N, H, D] (got %s)" % (tuple(k.shape),))
    H, D = k.shape[-2], k.shape[-1] * (2 if fp4 else 1)
    if D % MX_BLOCK:
        raise ValueError("a cache's head size must be a multiple of %d (got %d)" % (MX_BLOCK, D))
    codes, scales = k.shape, k.shape[:-1] + (D // MX_BLOCK,)
    dtype, byte, index = torch.uint8 if fp4 else torch.float8_e4m3fn, torch.uint8, k.get_device()
    # the usual case in few steps; what fails here is looked at one by one below
    if (index >= 0 and index == v.get_device() == k_scale.get_device() == v_scale.get_device() and
            k.dtype == v.dtype == dtype and k_scale.dtype == v_scale.dtype == byte and v.shape == codes and
            k_scale.shape == scales and v_scale.shape == scales and k.is_contiguous() and v.is_contiguous() and
            k_scale.is_contiguous() and v_scale.is_contiguous()):
        return codes[:-2], H, D, 0
    for name, t, dt, shape in (("k", k, dtype, codes), ("k_scale", k_scale, byte, scales), ("v", v, dtype, codes),
                               ("v_scale", v_scale, byte, scales)):
        if not t.is_cuda:
            raise ValueError("%s must be a device tensor (got %s)" % (name, t.device))
        if t.dtype != dt:
            raise TypeError("%s must be %s (got %s)" % (name, dt, t.dtype))
        if t.shape != shape:
            raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    _same_device(k, k_scale=k_scale, v=v, v_scale=v_scale)
    rooms = [_packed_tokens(t, n) for n, t in (("k", k), ("k_scale", k_scale), ("v", v), ("v_scale", v_scale))]
    if any(r != rooms[0] for r in rooms):
        raise ValueError("the slots of a cache's tensors must lie equally far apart")
    return codes[:-2], H, D, rooms[0]


def _is_fp4(k):
    if not isinstance(k, torch.Tensor) or k.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("a cache's k must be uint8 (MXFP4) or float8_e4m3fn (MXFP8)")
    return k.dtype == torch.uint8


def cache_write(k, v, k_cache, k_scale, v_cache, v_scale, *, k_len=None, cu_new=None, cu_k=None, max_new=None,
                max_k=None, stream=None) -> None:
    """Quantises new keys and values into an MXFP4 or MXFP8 cache (cache_empty), in place.

    k, v: [B, n, H, D] (or [B, F, N, H, D], or packed [T, H, D] with cu_new), bf16 or
    fp32, heads packed and tokens evenly apart; the cache [B, L, H, ...] (or a slice
    k_cache[:, :n] of longer slots, or packed with cu_k, default cu_new).  The new
    tokens become the last of their sequence's k_len[s] positions (int32 [n_seq], the
    new tokens counted; None: all L).  The queries of attention_fwd_fp4 and _fp8 with
    the same k_len lie at the same positions while k_len[s] <= L.  Tokens that fall
    outside the slot are dropped without a word (lengths stay on the device), and
    attention then takes a k_len[s] past L as L: check lengths where they are made.
    """
    fp4 = _is_fp4(k_cache)
    lead, H, D, room = _cache_args(k_cache, k_scale, v_cache, v_scale, fp4)
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if not t.is_cuda:
            raise ValueError("%s must be a device tensor (got %s)" % (name, t.device))
    shape = k.shape
    dims = len(shape)
    if not 3 <= dims <= 5 or v.shape != shape or shape[-2:] != (H, D):
        raise ValueError("k and v must be [..., %d, %d], alike (got %s, %s)" % (H, D, tuple(shape), tuple(v.shape)))
    if v.dtype != k.dtype:
        raise TypeError("v must be %s (got %s)" % (k.dtype, v.dtype))
    io = _io(k.dtype, "k and v")
    ldk = ldv = 0
    if not (k.is_contiguous() and v.is_contiguous()):
        (ldk, rk), (ldv, rv) = _token_strides(k, "k"), _token_strides(v, "v")
        if rk or rv:
            raise ValueError("k and v must have packed heads and evenly spaced tokens")
    if (dims == 3) != (len(lead) == 1):
        raise ValueError("packed k [T, H, D] go with a packed cache")
    if dims == 3:
        if cu_new is None:
            raise ValueError("packed k [T, H, D] needs cu_new")
        cu_k = cu_new if cu_k is None else cu_k
        n_seq = cu_new.numel() - 1
        if n_seq < 0:
            raise ValueError("cu_new must hold n_seq + 1 offsets")
        _check(cu_new, "cu_new", torch.int32, (n_seq + 1,))
        _check(cu_k, "cu_k", torch.int32, (n_seq + 1,))
        tn, tk = shape[0], lead[0]
        max_new = tn if max_new is None else min(int(max_new), tn)
        max_k = tk if max_k is None else min(int(max_k), tk)
    else:
        if cu_new is not None or cu_k is not None or max_new is not None or max_k is not None:
            raise ValueError("cu_new, cu_k, max_new and max_k belong to packed k [T, H, D]")
        n_seq = shape[0]
        if lead[0] != n_seq:
            raise ValueError("k and the cache must have the same batch size")
        max_new, max_k = shape[1:-2].numel(), lead[1:].numel()
        tn, tk = n_seq * max_new, n_seq * max_k
    if k_len is not None:
        _check(k_len, "k_len", torch.int32, (n_seq,))
    _same_device(k, v=v, k_cache=k_cache, cu_new=cu_new, cu_k=cu_k, k_len=k_len)
    desc = _lib.GdnCacheDesc(tn, tk, ldk, ldv, room, n_seq, H, D, max_new, max_k, io,
                             _lib.GDN_FP4_E2M1 if fp4 else _lib.GDN_FP8_E4M3)
    where, handle = _launch(stream, k.device)
    with where:
        st = _lib.load().gdn_cache_write(ctypes.byref(desc), k.data_ptr(), v.data_ptr(), _ptr(cu_new), _ptr(cu_k),
                                         _ptr(k_len), k_cache.data_ptr(), k_scale.data_ptr(), v_cache.data_ptr(),
                                         v_scale.data_ptr(), handle)
    if st != 0:
        raise GdnError(st, "gdn_cache_write")


def cache_read(k_cache, k_scale, v_cache, v_scale, *, dtype: torch.dtype = torch.bfloat16, k_len=None, cu_k=None,
               max_k=None, k=None, v=None, stream=None):
    """The values that a cache holds: (k, v) [..., H, D] in dtype (bf16 or fp32),
    contiguous.  Only the first k_len[s] places of each slot (None: all) are written;
    the others of k and v are left as they are (unset, where they are not given).
    Slots as for cache_write."""
    fp4 = _is_fp4(k_cache)
    lead, H, D, room = _cache_args(k_cache, k_scale, v_cache, v_scale, fp4)
    dtype = k.dtype if k is not None else v.dtype if v is not None else dtype
    io = _io(dtype, "k and v")
    shape = lead + (H, D)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _check(t, name, dtype, shape)
    if len(lead) == 1:
        if cu_k is None:
            raise ValueError("a packed cache needs cu_k")
        n_seq, tk = cu_k.numel() - 1, lead[0]
        if n_seq < 0:
            raise ValueError("cu_k must hold n_seq + 1 offsets")
        _check(cu_k, "cu_k", torch.int32, (n_seq + 1,))
        max_k = tk if max_k is None else min(int(max_k), tk)
    else:
        if cu_k is not None or max_k is not None:
            raise ValueError("cu_k and max_k belong to a packed cache")
        n_seq, max_k = lead[0], lead[1:].numel()
        tk = n_seq * max_k
    if k_len is not None:
        _check(k_len, "k_len", torch.int32, (n_seq,))
    _same_device(k_cache, cu_k=cu_k, k_len=k_len, k=k, v=v)
    desc = _lib.GdnCacheDesc(0, tk, 0, 0, room, n_seq, H, D, 0, max_k, io,
                             _lib.GDN_FP4_E2M1 if fp4 else _lib.GDN_FP8_E4M3)
    where, handle = _launch(stream, k_cache.device)
    with where:   # allocations belong to the launch stream
        k = k_cache.new_empty(shape, dtype=dtype) if k is None else k
        v = k_cache.new_empty(shape, dtype=dtype) if v is None else v
        st = _lib.load().gdn_cache_read(ctypes.byref(desc), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale),
                                        _ptr(cu_k), _ptr(k_len), _ptr(k), _ptr(v), handle)
    if st != 0:
        raise GdnError(st, "gdn_cache_read")
    return k, v


def _attention_mx(fp4, q, k, k_scale, v, v_scale, causal, causal_block, scale, cu_q, cu_k, max_q, max_k, k_len, o, lse,
                  return_lse, workspace, stream):
    lead, Hk, D, room = _cache_args(k, k_scale, v, v_scale, fp4)
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if not q.is_cuda:
        raise ValueError("q must be a device tensor (got %s)" % q.device)
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be %s (got %s)" % (torch.bfloat16, q.dtype))
    shape = q.shape
    dims = len(shape)
    if not 3 <= dims <= 5 or shape[-1] != D or (dims == 3) != (len(lead) == 1):
        raise ValueError("q must be [B, L, H, %d] or [B, F, N, H, %d], or packed [T, H, %d] over a packed cache (got %s)"
                         % (D, D, D, tuple(shape)))
    Hq = shape[-2]
    ldq, rq = (0, 0) if q.is_contiguous() else _token_strides(q, "q")
    if rq:
        raise ValueError("q must have packed heads and evenly spaced tokens")
    if dims == 3:
        if cu_q is None:
            raise ValueError("packed q [T, H, D] needs cu_q")
        cu_k = cu_q if cu_k is None else cu_k
        n_seq = cu_q.numel() - 1
        if n_seq < 0:
            raise ValueError("cu_q must hold n_seq + 1 offsets")
        _check(cu_q, "cu_q", torch.int32, (n_seq + 1,))
        _check(cu_k, "cu_k", torch.int32, (n_seq + 1,))
        tq, tk = shape[0], lead[0]
        max_q = tq if max_q is None else min(int(max_q), tq)
        max_k = tk if max_k is None else min(int(max_k), tk)
    else:
        if cu_q is not None or cu_k is not None or max_q is not None or max_k is not None:
            raise ValueError("cu_q, cu_k, max_q and max_k belong to packed q [T, H, D]")
        n_seq = shape[0]
        if lead[0] != n_seq:
            raise ValueError("q and the cache must have the same batch size")
        max_q, max_k = shape[1:-2].numel(), lead[1:].numel()
        tq, tk = n_seq * max_q, n_seq * max_k
    if causal_block is None:
        causal_block = shape[2] if dims == 5 else 1
    if k_len is not None:
        _check(k_len, "k_len", torch.int32, (n_seq,))
    if o is not None:
        _check(o, "o", q.dtype, shape)
    if lse is not None:
        _check(lse, "lse", torch.float32, shape[:-1])
    device = q.device
    if workspace is not None:
        _check_workspace(workspace, device)
    _same_device(q, k=k, cu_q=cu_q, cu_k=cu_k, k_len=k_len, o=o, lse=lse)
    desc = _lib.GdnAttnDesc(tq, tk, ldq, 0, 0, room, n_seq, Hq, Hk, D, max_q, max_k, min(int(causal_block), 2 ** 31 - 1),
                            _lib.GDN_FP4_E2M1 if fp4 else _lib.GDN_FP8_E4M3,
                            _lib.GDN_FLAG_ATTN_CAUSAL if causal else 0, D ** -0.5 if scale is None else scale)
    lib = _lib.load()
    fn = lib.gdn_attn_fwd_fp4 if fp4 else lib.gdn_attn_fwd_fp8
    where, handle = _launch(stream, device)
    with where:   # allocations belong to the launch stream
        if o is None:
            o = q.new_empty(shape)
        if lse is None and return_lse:
            lse = q.new_empty(shape[:-1], dtype=torch.float32)
        if workspace is None:
            need = lib.gdn_attn_workspace_size(ctypes.byref(desc))
            workspace = q.new_empty(need, dtype=torch.uint8) if need else None
        st = fn(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), k_scale.data_ptr(), v.data_ptr(), v_scale.data_ptr(),
                _ptr(cu_q), _ptr(cu_k), _ptr(k_len), o.data_ptr(), _ptr(lse), _ptr(workspace), _ws_bytes(workspace),
                handle)
    if st != 0:
        raise GdnError(st, "gdn_attn_fwd_fp4" if fp4 else "gdn_attn_fwd_fp8")
    return o, lse


def attention_fwd_fp4(q, k, k_scale, v, v_scale, *, causal: bool = False, causal_block: Optional[int] = None,
                      scale=None, cu_q=None, cu_k=None, max_q=None, max_k=None, k_len=None, o=None, lse=None,
                      return_lse: bool = True, workspace=None, stream=None):
    """attention_fwd over keys and values in MXFP4 (cache_write).

    q: bf16 [B, L, Hq, D], [B, F, N, Hq, D] or packed [T, Hq, D]; k, v: uint8
    [B, Lk, Hk, D/2] (two E2M1 codes a byte) with k_scale, v_scale uint8
    [B, Lk, Hk, D/32], or packed; tokens packed, slices k[:, :n] of longer slots will
    do.  D in {32, 64, 128}.  The rest as for attention_fwd; forward only, no gradient.

    Kernel and splits of the keys are chosen by the bounds of the call alone, so give
    packed calls max_q and max_k: max_q Hq / Hk <= 32 takes the kernel for few rows and
    splits the keys finely, without max_q that is all tokens.  A long prompt and single
    tokens on long caches are better two calls (eight single queries on caches of 40 to
    32768 keys, 32 / 8 heads: 31 us alone, 541 in one call with a prompt of 512).
    """
    return _attention_mx(True, q, k, k_scale, v, v_scale, causal, causal_block, scale, cu_q, cu_k, max_q, max_k, k_len,
                         o, lse, return_lse, workspace, stream)


def attention_fwd_fp8(q, k, k_scale, v, v_scale, *, causal: bool = False, causal_block: Optional[int] = None,
                      scale=None, cu_q=None, cu_k=None, max_q=None, max_k=None, k_len=None, o=None, lse=None,
                      return_lse: bool = True, workspace=None, stream=None):
    """attention_fwd_fp4 over keys and values in MXFP8: k, v float8_e4m3fn
    [B, Lk, Hk, D], scales as there."""
    return _attention_mx(False, q, k, k_scale, v, v_scale, causal, causal_block, scale, cu_q, cu_k, max_q, max_k, k_len,
                         o, lse, return_lse, workspace, stream)
