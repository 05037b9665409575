"""A training step: attention of packed sequences with its gradients, and activations kept in 8 bits.  Same manner as
``stack.py``: the compiled module ``_gdn_torch`` checks the tensors, allocates outputs and passes raw pointers and the
current stream to libgdn (``include/gdn.h``)."""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import load_library, stack

__all__ = ["gdn_attention_fwd", "gdn_attention_bwd", "attention", "attention_bwd_workspace_size", "gdn_act8_save",
           "gdn_act8_load", "linear8", "ACT8_GROUP"]

#: Elements of a row that share a scale.
ACT8_GROUP = 128


# ----------------------------------------------------- activations in 8 bits
def gdn_act8_save(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """8-bit codes of x bf16 [..., D] (dense, or with a longer stride between its tokens): (codes float8_e4m3fn [..., D],
    scale fp32 [..., ceil(D / 128)]), one power of two for each 128 elements of a row.  See include/gdn.h."""
    return (stack._c or stack._load()).act8_save(x, codes, scale)


def gdn_act8_load(codes: torch.Tensor, scale: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that codes and scales stand for, bf16 [..., D]."""
    return (stack._c or stack._load()).act8_load(codes, scale, out)


class _Linear8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight):
        y, kept = x @ weight.T, ()
        if ctx.needs_input_grad[1]:
            rows = x.reshape(-1, x.shape[-1])  # (a copy where they have no single stride)
            kept = gdn_act8_save(rows if rows.stride(1) == 1 else rows.contiguous())
        ctx.save_for_backward(weight, *kept)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        weight, *kept = ctx.saved_tensors
        dx = dy @ weight if ctx.needs_input_grad[0] else None
        dw = dy.reshape(-1, dy.shape[-1]).T @ gdn_act8_load(*kept).view(-1, weight.shape[1]) if kept else None
        return dx, dw


def linear8(x: torch.Tensor, weight: torch.Tensor) -> torch.Tensor:
    """x @ weight.T (x bf16 [..., in] of any strides, weight bf16 [out, in]), differentiable once, that keeps x in 8 bits for
    the weight's gradient."""
    return _Linear8.apply(x, weight)


# -------------------------------------------------------------- attention


def gdn_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                      cu_seqlens_k: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
                      o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      dev_status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax attention of packed sequences: see include/gdn.h.

    q bf16 [Tq, HQ, D], k, v bf16 [Tk, HK, D] (from 16-byte boundaries on, any token stride that is a multiple of 8), HQ a multiple of HK, D 64 or
    128; cu_seqlens int32 [N + 1] (None: one sequence), cu_seqlens_k the keys' offsets where they are others (then the
    last row of a sequence sees all of its keys under ``causal``).  Returns (o bf16 [Tq, HQ, D], lse fp32 [Tq, HQ])."""
    return (stack._c or stack._load()).attention_fwd(q, k, v, cu_seqlens, cu_seqlens_k, 1 if causal else 0,
                                                     -1.0 if scale is None else scale, o, lse, dev_status)


def attention_bwd_workspace_size(N, Tq, Tk, HQ, HK, D) -> int:
    """Bytes of workspace that gdn_attention_bwd needs for these sizes, enough for all smaller ones too."""
    return int(load_library().gdn_attention_bwd_workspace_size(N, Tq, Tk, HQ, HK, D))


def gdn_attention_bwd(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                      cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
                      causal: bool = True, scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                      dev_status: Optional[torch.Tensor] = None):
    """Gradients of gdn_attention_fwd: do, o bf16 [Tq, HQ, D] and lse fp32 [Tq, HQ] as it returned them, the rest as it
    took them.  Returns (dq, dk, dv), bf16 and dense."""
    return (stack._c or stack._load()).attention_bwd(do, q, k, v, o, lse, cu_seqlens, cu_seqlens_k, 1 if causal else 0,
                                                     -1.0 if scale is None else scale, workspace, dev_status)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, cu_seqlens_k, causal, scale, dev_status):
        o, lse = gdn_attention_fwd(q, k, v, cu_seqlens=cu_seqlens, cu_seqlens_k=cu_seqlens_k, causal=causal, scale=scale,
                                   dev_status=dev_status)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, cu_seqlens_k)
        ctx.args = (causal, scale, dev_status)  # (the status is the caller's to clear meanwhile)
        return o

    @staticmethod
    @once_differentiable  # the gradient kernels have no gradient of their own: a second derivative is an error
    def backward(ctx, do):
        q, k, v, o, lse, cu, cu_k = ctx.saved_tensors
        causal, scale, status = ctx.args
        dq, dk, dv = gdn_attention_bwd(stack._gradient(do), q, k, v, o, lse, cu_seqlens=cu, cu_seqlens_k=cu_k, causal=causal,
                                       scale=scale, dev_status=status)
        return dq, dk, dv, None, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
              cu_seqlens_k: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
              dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable (once) gdn_attention_fwd; returns o.  The forward keeps q, k, v, o and lse for the gradient.  Both
    directions report to ``dev_status`` what they could not do (offsets that break the rules: rows of that sequence are not
    written, in the gradients neither)."""
    return _Attention.apply(q, k, v, cu_seqlens, cu_seqlens_k, causal, scale, dev_status)
