"""torch.autograd bindings of the frame scan and of the operators around it
(argument marshalling only).

``frame_scan(q, k, v, beta, alpha, S0=None, ...)`` returns (o, S_final) as a
differentiable function of every tensor input: the forward pass is
gdn_frame_scan_fwd_save, which keeps each frame's operands for the backward
pass (gdn_saved_size bytes, held by the autograd graph until backward runs or
the graph is freed), and the backward pass is gdn_frame_scan_bwd_saved.  With
``recompute=True`` the forward pass keeps nothing and the backward pass
(gdn_frame_scan_bwd) recomputes the operands instead.  Both give the same
gradients bit for bit.

``layer_norm``, ``rotary`` and ``attention`` are differentiable once.  A training
step captured into a graph takes its leaves' first gradients inside the capture:
torch ties a leaf's accumulation to the stream of the first graph that uses it,
so no eager graph of the same leaves may be alive meanwhile.  Where one has to
be, capture the api calls (layer_norm_fwd, layer_norm_bwd and so on) instead.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import api


class _FrameScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, alpha, S0, gates_are_logits, eps, normalize_keys, reverse, recompute):
        kw = dict(gates_are_logits=gates_are_logits, eps=eps, normalize_keys=normalize_keys, reverse=reverse)
        if recompute:
            o, S_final = api.frame_scan_fwd(q, k, v, beta, alpha, S0, **kw)
            saved = None
        else:
            o, S_final, saved = api.frame_scan_fwd_save(q, k, v, beta, alpha, S0, **kw)
        ctx.kw = kw
        ctx.has_S0 = S0 is not None
        ctx.saved_buf = saved
        # S0 is needed by the recomputing backward only (the saved buffer holds its copy)
        ctx.save_for_backward(q, k, v, beta, alpha, S0 if (recompute and S0 is not None) else None)
        return o, S_final

    @staticmethod
    def backward(ctx, dO, dS_final):
        q, k, v, beta, alpha, S0 = ctx.saved_tensors
        dO = torch.zeros_like(q) if dO is None else dO.contiguous().to(q.dtype)
        dS_final = None if dS_final is None else dS_final.contiguous().float()
        dq, dk, dv, dbeta, dalpha, dS0 = api.frame_scan_bwd(q, k, v, beta, alpha, dO, S0, dS_final,
                                                            return_dS0=ctx.has_S0, saved=ctx.saved_buf, **ctx.kw)
        ctx.saved_buf = None
        return dq, dk, dv, dbeta, dalpha, dS0, None, None, None, None, None


def frame_scan(q, k, v, beta, alpha, S0=None, *, gates_are_logits: bool = False, eps: float = 1e-6,
               normalize_keys: bool = True, reverse: bool = False, recompute: bool = False):
    """Differentiable whole-clip scan: (o, S_final) with gradients to q, k, v,
    beta, alpha and S0 (layouts as for api.frame_scan_fwd)."""
    return _FrameScan.apply(q, k, v, beta, alpha, S0, gates_are_logits, eps, normalize_keys, reverse, recompute)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = api.layer_norm_fwd(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, mean, rstd, weight, bias)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight, bias = ctx.saved_tensors
        dx, dweight, dbias = api.layer_norm_bwd(dy.contiguous(), x, mean, rstd, weight, bias)
        return dx, dweight, dbias, None


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-6):
    """Differentiable layer norm over the last axis (layouts as for
    api.layer_norm_fwd); keeps each row's mean and rstd for the backward pass."""
    return _LayerNorm.apply(x, weight, bias, eps)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, pos, axes, theta, halves, inverse):
        ctx.save_for_backward(pos)
        ctx.kw = dict(axes=axes, theta=theta, halves=halves, inverse=not inverse)
        return api.rotary(q, k, pos, axes=axes, theta=theta, halves=halves, inverse=inverse)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        pos, = ctx.saved_tensors
        dq = None if dq is None else dq.contiguous()
        dk = None if dk is None else dk.contiguous()
        if dq is not None or dk is not None:
            dq, dk = api.rotary(dq, dk, pos, **ctx.kw)
        return dq, dk, None, None, None, None, None


def rotary(q, k, pos, *, axes, theta: float = 10000.0, halves: bool = False, inverse: bool = False):
    """Differentiable rotary positions (layouts as for api.rotary); the gradient
    is the rotation turned back.  Positions take no gradient: a pos that asks for
    one is refused while gradients are recorded."""
    if getattr(pos, "requires_grad", False) and torch.is_grad_enabled():
        raise ValueError("positions take no gradient: pass pos.detach()")
    return _Rotary.apply(q, k, pos, tuple(axes), theta, halves, inverse)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, causal_block, scale, cu_q, cu_k, max_q, max_k):
        kw = dict(causal=causal, causal_block=causal_block, scale=scale, max_q=max_q, max_k=max_k)
        # tokens of no sequence: zeros, so that they add nothing further on
        o = None if cu_q is None else torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        o, lse = api.attention_fwd(q, k, v, cu_q=cu_q, cu_k=cu_k, o=o, **kw)
        ctx.kw = kw
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_k)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dO):
        q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
        outs = [None] * 3 if cu_q is None else [torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v)]
        dq, dk, dv = api.attention_bwd(q, k, v, o, lse, dO.contiguous(), cu_q=cu_q, cu_k=cu_k, dq=outs[0], dk=outs[1],
                                       dv=outs[2], **ctx.kw)
        return dq, dk, dv, None, None, None, None, None, None, None


def attention(q, k, v, *, causal: bool = False, causal_block=None, scale=None, cu_q=None, cu_k=None, max_q=None,
              max_k=None):
    """Differentiable softmax attention (layouts as for api.attention_fwd); keeps
    o and the logarithm of each row's sum for the backward pass.  Tokens of no
    packed sequence give zeros, in the output and in the gradients."""
    return _Attention.apply(q, k, v, causal, causal_block, scale, cu_q, cu_k, max_q, max_k)
