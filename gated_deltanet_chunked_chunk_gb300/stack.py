"""Around the recurrence: norms with a gate and a residual, rotary positions, and the paged 8-bit cache with the
attention that reads it.  Same manner as the rest of the binding: arguments are checked, outputs allocated, raw
pointers and the current stream passed to libgdn (``include/gdn.h``); here that is done by the compiled module
``_gdn_torch`` (``csrc/gdn_torch.cpp``), since a decode step's calls take less time on the GPU than the same checks do
in Python.  TypeError: a wrong type; ValueError: a wrong device, shape or layout; GDNError: what the library refuses;
torch.OutOfMemoryError: an output or a workspace that does not fit."""
from __future__ import annotations

import functools
import importlib.machinery
import importlib.util
import math
import os
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import GDNError, lib_path, load_library

__all__ = ["gdn_norm_gate", "gdn_norm_gate_bwd", "norm_gate", "gdn_norm_gate_save8", "gdn_norm_gate_bwd8", "gdn_rope",
           "rotary_embedding", "rope_frequencies",
           "gdn_paged_plan", "gdn_kv8_append", "gdn_kv8_attention", "kv8_attention_workspace_size", "KV8_PAGE_SIZES",
           "KV8_EXP_MIN"]

#: Page sizes that the attention takes.
KV8_PAGE_SIZES = (16, 32, 64, 128)
#: Lowest exponent of a page's scale.
KV8_EXP_MIN = -60

_ACT = {None: 0, "none": 0, "silu": 1, "swish": 1, "sigmoid": 2}
_c = None


def _load():
    """The compiled binding (built by ``build.py``); raises if it is missing or was built for another interpreter or
    PyTorch, whose tensors it would misread."""
    global _c
    from . import build
    load_library()
    path = os.path.join(os.path.dirname(lib_path()), "_gdn_torch.so")
    if not os.path.exists(path):
        raise RuntimeError(f"_gdn_torch.so not found at {path}; build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    if not build.binding_fits():
        raise RuntimeError(f"{path} was built for another interpreter or PyTorch than the running one; build it again "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    loader = importlib.machinery.ExtensionFileLoader(__package__ + "._gdn_torch", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location(loader.name, path, loader=loader))
    loader.exec_module(module)
    module.set_errors(GDNError, torch.OutOfMemoryError)
    _c = module
    return module


def _act_of(activation, fn):
    try:
        return _ACT[activation]
    except (KeyError, TypeError):
        raise ValueError(f"{fn}: activation must be None, 'silu' or 'sigmoid', got {activation!r}") from None


# ------------------------------------------------------------------- norms
def gdn_norm_gate(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                  z: Optional[torch.Tensor] = None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0,
                  y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """RMS norm with a gate and a scaled residual over the last dimension: h = residual + res_scale x (x alone without
    one, whatever res_scale is), y = h / sqrt(mean(h^2) + eps) * weight * act(z).

    x, residual bf16 [..., D]; weight fp32 [D]; z bf16 of x's shape, dense or with a longer stride between its tokens
    (a slice of a projection); activation 'silu' or 'sigmoid' (used where z is given).  Returns (y, h), h None
    without a residual.  ``y`` / ``h`` may be given, x and residual themselves among them."""
    return (_c or _load()).norm_gate(x, weight, residual, z, _act_of(activation, "gdn_norm_gate"), eps, res_scale, y, h)


def gdn_norm_gate_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, z: Optional[torch.Tensor] = None,
                      dh: Optional[torch.Tensor] = None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0,
                      workspace: Optional[torch.Tensor] = None):
    """Gradients of gdn_norm_gate: dy, h (what was normed) bf16 [..., D], dh the gradient that reaches h from its other
    uses (None without a residual).  Returns (dx, dresidual, dz, dweight): bf16 but the fp32 dweight [D]; dresidual
    None without dh, dz None without z.  dx is res_scale times the gradient of h whether dh is there or not; the form
    without a residual, whose forward does not use res_scale, has its gradient with res_scale = 1."""
    return (_c or _load()).norm_gate_bwd(dy, h, weight, z, dh, _act_of(activation, "gdn_norm_gate_bwd"), eps, res_scale,
                                         workspace)


class _NormGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, z, activation, eps, res_scale):
        y, h = gdn_norm_gate(x, weight, residual=residual, z=z, activation=activation, eps=eps, res_scale=res_scale)
        ctx.save_for_backward(x if h is None else h, weight, z)
        # the forward scales x only where a residual is added to it
        ctx.args = (activation, eps, 1.0 if residual is None else res_scale, residual is not None)
        return y if h is None else (y, h)

    @staticmethod
    @once_differentiable  # the gradient kernels have no gradient of their own: a second derivative is an error
    def backward(ctx, dy, dh=None):
        h, weight, z = ctx.saved_tensors
        activation, eps, res_scale, has_res = ctx.args
        if has_res:
            dh = torch.zeros_like(h) if dh is None else dh.to(torch.bfloat16).contiguous()
        dx, dres, dz, dw = gdn_norm_gate_bwd(dy.to(torch.bfloat16).contiguous(), h, weight, z=z, dh=dh if has_res else None,
                                             activation=activation, eps=eps, res_scale=res_scale)
        return dx, dw, dres, dz, None, None, None


def gdn_norm_gate_save8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0):
    """gdn_norm_gate that also writes 8-bit codes of what its backward needs (``gdn_act8_save``): returns (y, h, h_codes,
    h_scale, z_codes, z_scale), the last two None without a gate.  D a multiple of 8, at most 16384."""
    return (_c or _load()).norm_gate_save8(x, weight, residual, z, _act_of(activation, "gdn_norm_gate_save8"), eps, res_scale)


def gdn_norm_gate_bwd8(dy: torch.Tensor, h_codes: torch.Tensor, h_scale: torch.Tensor, weight: torch.Tensor,
                       z_codes: Optional[torch.Tensor] = None, z_scale: Optional[torch.Tensor] = None,
                       dh: Optional[torch.Tensor] = None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0,
                       workspace: Optional[torch.Tensor] = None):
    """gdn_norm_gate_bwd at the values that the codes of gdn_norm_gate_save8 stand for; the same results, (dx, dresidual,
    dz, dweight)."""
    return (_c or _load()).norm_gate_bwd8(dy, h_codes, h_scale, weight, z_codes, z_scale, dh,
                                          _act_of(activation, "gdn_norm_gate_bwd8"), eps, res_scale, workspace)


def _gradient(t):
    """An arriving gradient as the kernels take it: bf16, dense, on a 16-byte boundary (a piece of a wider one may start anywhere)."""
    t = t.to(torch.bfloat16).contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _on_boundary(t, strides=False):
    """An input as the kernels with codes take it: from a 16-byte boundary on and, with ``strides``, in steps of 8 elements."""
    if not torch.is_tensor(t) or (t.data_ptr() % 16 == 0 and not (strides and any(s % 8 for s in t.stride()[:-1]))):
        return t
    return t.clone(memory_format=torch.contiguous_format) if t.is_contiguous() else t.contiguous() if strides else t


class _NormGate8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, z, activation, eps, res_scale):
        args = dict(activation=activation, eps=eps, res_scale=res_scale)
        ctx.fused = not torch.is_tensor(x) or (x.dim() > 0 and x.shape[-1] % 8 == 0 and x.shape[-1] <= 16384)
        if ctx.fused:
            y, h, *codes = gdn_norm_gate_save8(_on_boundary(x), weight, residual=_on_boundary(residual), z=_on_boundary(z, True), **args)
        else:  # a width that only gdn_norm_gate takes
            y, h = gdn_norm_gate(x, weight, residual=residual, z=z, **args)
            save = (_c or _load()).act8_save
            codes = save(x if h is None else h, None, None) + ((None, None) if z is None else save(z, None, None))
        ctx.save_for_backward(weight, *codes)
        ctx.args = (activation, eps, 1.0 if residual is None else res_scale, residual is not None)
        return y if h is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        weight, h8, hs, z8, zs = ctx.saved_tensors
        activation, eps, res_scale, has_res = ctx.args
        dy = _gradient(dy)
        if has_res:
            dh = torch.zeros_like(dy) if dh is None else _gradient(dh)
        args = dict(dh=dh if has_res else None, activation=activation, eps=eps, res_scale=res_scale)
        if ctx.fused:
            dx, dres, dz, dw = gdn_norm_gate_bwd8(dy, h8, hs, weight, z_codes=z8, z_scale=zs, **args)
        else:
            load = (_c or _load()).act8_load
            dx, dres, dz, dw = gdn_norm_gate_bwd(dy, load(h8, hs, None), weight, z=None if z8 is None else load(z8, zs, None), **args)
        return dx, dw, dres, dz, None, None, None


def norm_gate(x, weight, residual=None, z=None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0, save8: bool = False):
    """Differentiable (once) gdn_norm_gate: returns (y, h), h None without a residual; gradients for x, weight, residual, z.
    With ``save8`` the forward keeps 8-bit codes of h and z for the gradient instead of the tensors themselves: in the same pass
    for widths that are a multiple of 8 and at most 16384 (inputs that do not lie as gdn_norm_gate_save8 wants are copied), in
    passes of their own for others."""
    out = (_NormGate8 if save8 else _NormGate).apply(x, weight, residual, z, activation, eps, res_scale)
    return out if isinstance(out, tuple) else (out, None)


# ------------------------------------------------------------------ rotary
def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original_max_position: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device=None) -> Tuple[torch.Tensor, float]:
    """(inv_freq fp32 [rotary_dim / 2], attention_factor) for gdn_rope, formed in 64 bits.

    scaling, for contexts ``factor`` times the trained length: None; 'linear' (all angles / factor); 'ntk' (a larger
    base, such that the slowest pair turns factor times slower and the fastest as before); 'yarn' (pairs that turn more
    than beta_fast times in original_max_position stay, those that turn less than beta_slow times are slowed by
    factor, a linear ramp between them, and the logits' temperature goes into attention_factor = 0.1 ln(factor) + 1)."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and at least 2, got {rotary_dim}")
    if not (base > 0 and math.isfinite(base)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("rope_frequencies: base > 0 and factor >= 1 are needed")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim
    if scaling is None:
        inv, att = base ** -i, 1.0
    elif scaling == "linear":
        inv, att = base ** -i / factor, 1.0
    elif scaling == "ntk":
        grown = base * factor ** (rotary_dim / (rotary_dim - 2)) if rotary_dim > 2 else base
        inv, att = grown ** -i, 1.0
    elif scaling == "yarn":
        inv = base ** -i
        place = [rotary_dim * math.log(original_max_position / (b * 2 * math.pi)) / (2 * math.log(base))
                 for b in (beta_fast, beta_slow)]  # the pair that turns b times in the trained length
        lo, hi = max(math.floor(place[0]), 0), min(math.ceil(place[1]), rotary_dim - 1)
        ramp = ((torch.arange(rotary_dim // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv = inv / factor * ramp + inv * (1 - ramp)
        att = 0.1 * math.log(factor) + 1.0
    else:
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    return inv.float().to(device) if device is not None else inv.float(), att


def gdn_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, inv_freq: torch.Tensor,
             interleaved: bool = False, attention_factor: float = 1.0, inverse: bool = False,
             q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Rotary positions: q bf16 [T, HQ, D], k bf16 [T, HK, D] or None (any token stride), positions int32 [T], inv_freq
    fp32 [rotary_dim / 2].  ``interleaved`` pairs neighbours, else the halves of the rotated part; ``inverse`` turns
    back (the gradient).  Returns (q_out, k_out), dense; q and k themselves may be given for them where dense."""
    return (_c or _load()).rope(q, k, positions, inv_freq, 1 if interleaved else 0, 1 if inverse else 0, attention_factor,
                                q_out, k_out)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, interleaved, attention_factor):
        ctx.save_for_backward(positions, inv_freq)
        ctx.args = (interleaved, attention_factor)
        return gdn_rope(q, k, positions, inv_freq, interleaved=interleaved, attention_factor=attention_factor)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        positions, inv_freq = ctx.saved_tensors
        interleaved, factor = ctx.args
        dk = None if dk is None else dk.to(torch.bfloat16).contiguous()
        dq, dk = gdn_rope(dq.to(torch.bfloat16).contiguous(), dk, positions, inv_freq, interleaved=interleaved,
                          attention_factor=factor, inverse=True)
        return dq, dk, None, None, None, None


def rotary_embedding(q, k, positions, inv_freq, interleaved: bool = False, attention_factor: float = 1.0):
    """Differentiable (once) gdn_rope of q and k (k may be None)."""
    return _Rotary.apply(q, k, positions, inv_freq, interleaved, attention_factor)


# ------------------------------------------------------------- paged cache
def gdn_paged_plan(cached_lens: torch.Tensor, cu_seqlens: torch.Tensor, block_table: torch.Tensor,
                   free_pages: torch.Tensor, num_free: torch.Tensor, page_size: int, num_tokens: int,
                   dev_status: Optional[torch.Tensor] = None):
    """Pages, slots and positions of one step: see include/gdn.h.  cached_lens int32 [N], cu_seqlens int32 [N + 1],
    block_table int32 [N, width] (entries of new pages written in place), free_pages int32 [F], num_free int32 [1],
    num_tokens = cu_seqlens[N] (a host number, so nothing is read back).  Returns (seq_lens [N], slot_mapping [T],
    positions [T], num_free_out [1]), all int32."""
    return (_c or _load()).paged_plan(cached_lens, cu_seqlens, block_table, free_pages, num_free, page_size, num_tokens,
                                      dev_status)


def gdn_kv8_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   k_scale: torch.Tensor, v_scale: torch.Tensor, slot_mapping: torch.Tensor,
                   dev_status: Optional[torch.Tensor] = None) -> None:
    """New keys and values into the 8-bit cache, in place.  k, v bf16 [T, HK, D] (any token stride); k_cache, v_cache
    float8_e4m3fn [P, HK, page_size, D]; k_scale, v_scale fp32 [P, HK]; slot_mapping int32 [T] (-1 skips a token)."""
    (_c or _load()).kv8_append(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, dev_status)


@functools.lru_cache(maxsize=256)
def kv8_attention_workspace_size(N, T, HQ, HK, D, max_q_len, max_seq_len) -> int:
    """Bytes of workspace that gdn_kv8_attention needs for these sizes."""
    return int(load_library().gdn_kv8_attention_workspace_size(N, T, HQ, HK, D, max_q_len, max_seq_len))


def gdn_kv8_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                      v_scale: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      cu_seqlens: Optional[torch.Tensor] = None, max_q_len: int = 1,
                      max_seq_len: Optional[int] = None, scale: Optional[float] = None,
                      o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention over the paged 8-bit cache: see include/gdn.h.

    q bf16 [T, HQ, D] (any token stride), the cache as gdn_kv8_append writes it, block_table int32 [N, width], seq_lens
    int32 [N] (contexts, the new tokens among them), cu_seqlens int32 [N + 1] or None (one token a request).
    ``max_q_len`` and ``max_seq_len`` bound a request's new tokens and its context on the host (default: one token;
    all places of a table row).  ``lse`` (fp32 [T, HQ]), where given, receives the logsumexp.  Returns o bf16 [T, HQ, D]."""
    return (_c or _load()).kv8_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, max_q_len,
                                         -1 if max_seq_len is None else max_seq_len, -1.0 if scale is None else scale, o, lse,
                                         workspace, dev_status)
