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
_current_device = torch.cuda.current_device
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
