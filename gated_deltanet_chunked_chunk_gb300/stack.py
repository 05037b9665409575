"""Around the recurrence: norms with a gate and a residual, rotary positions, and the paged 8-bit cache with the
attention that reads it.  Same manner as the rest of the binding: arguments are checked, outputs allocated with
``torch.empty``, raw pointers and the current stream passed to libgdn (``include/gdn.h``)."""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import GDN_OK, GDNError, _check, load_library

__all__ = ["gdn_norm_gate", "gdn_norm_gate_bwd", "norm_gate", "gdn_rope", "rotary_embedding", "rope_frequencies",
           "gdn_paged_plan", "gdn_kv8_append", "gdn_kv8_attention", "kv8_attention_workspace_size", "KV8_PAGE_SIZES",
           "KV8_EXP_MIN"]

#: Page sizes that the attention takes.
KV8_PAGE_SIZES = (16, 32, 64, 128)
#: Lowest exponent of a page's scale.
KV8_EXP_MIN = -60

_BF, _F32, _I32, _F8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
_ACT = {None: 0, "none": 0, "silu": 1, "swish": 1, "sigmoid": 2}
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _need(t, name, dtype, dev, ndim):
    """A contiguous tensor of this type, device and rank; the calls below are on the path of single tokens, so the
    tests are the cheap ones and _check words the refusal."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or t.dim() != ndim or not t.is_contiguous():
        if t is None:
            raise TypeError(f"{name} is required")
        _check(t, name, dtype, dev, ndim)


def _rows_dense(t, name, dtype, dev, ndim):
    """A tensor whose last two dimensions are dense and whose first may have any stride; returns that stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and H > 1) or (s0 < H * D and T > 1):
        raise ValueError(f"{name}: the heads of a token must be dense (the library does not copy)")
    return s0 if T > 1 else H * D


def _raise(fn, rc):
    raise GDNError(fn, rc)


# ------------------------------------------------------------------- norms
def _gate_layout(z, x, fn):
    """(rows of z in a stretch, elements between stretches); (0, 0) for a dense z."""
    if z.dtype is not _BF:
        raise TypeError(f"z must be {_BF}, got {z.dtype}")
    if z.device != x.device:
        raise ValueError(f"z must be on {x.device}, got {z.device}")
    if z.shape != x.shape:
        raise ValueError(f"{fn}: z must have the shape of x, {tuple(x.shape)}")
    if z.is_contiguous():
        return 0, 0
    if z.dim() == 3 and z.stride(2) == 1 and z.stride(1) == z.shape[2]:
        return z.shape[1], z.stride(0)
    if z.dim() == 2 and z.stride(1) == 1:
        return 1, z.stride(0)
    raise ValueError(f"{fn}: z must be dense, or [tokens, heads, D] / [rows, D] with a longer stride between tokens")


def _act_of(activation, z, fn):
    if activation not in _ACT:
        raise ValueError(f"{fn}: activation must be None, 'silu' or 'sigmoid', got {activation!r}")
    if z is None:
        return 0
    act = _ACT[activation]
    if act == 0:
        raise ValueError(f"{fn}: a gate z needs an activation")
    return act


def gdn_norm_gate(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                  z: Optional[torch.Tensor] = None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0,
                  y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """RMS norm with a gate and a scaled residual over the last dimension: h = residual + res_scale x (x alone without
    one), y = h / sqrt(mean(h^2) + eps) * weight * act(z).

    x, residual bf16 [..., D]; weight fp32 [D]; z bf16 of x's shape, dense or with a longer stride between its tokens
    (a slice of a projection); activation 'silu' or 'sigmoid' (used where z is given).  Returns (y, h), h None
    without a residual.  ``y`` / ``h`` may be given, x and residual themselves among them."""
    dev = x.device
    _need(x, "x", _BF, dev, x.dim())
    D = x.shape[-1] if x.dim() else 0
    _need(weight, "weight", _F32, dev, 1)
    if D < 1 or weight.shape[0] != D:
        raise ValueError(f"gdn_norm_gate: weight must be [{D}], x [..., {D}]")
    act = _act_of(activation, z, "gdn_norm_gate")
    zr, zs = _gate_layout(z, x, "gdn_norm_gate") if act else (0, 0)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", _BF, dev, x.dim())
        if y.shape != x.shape:
            raise ValueError("gdn_norm_gate: y must have the shape of x")
    if residual is not None:
        _need(residual, "residual", _BF, dev, x.dim())
        if residual.shape != x.shape:
            raise ValueError("gdn_norm_gate: residual must have the shape of x")
        if h is None:
            h = torch.empty_like(x)
        else:
            _need(h, "h", _BF, dev, x.dim())
            if h.shape != x.shape:
                raise ValueError("gdn_norm_gate: h must have the shape of x")
    elif h is not None:
        raise ValueError("gdn_norm_gate: h is an output of the form with a residual")
    rc = load_library().gdn_norm_gate(
        x.data_ptr(), None if residual is None else residual.data_ptr(), z.data_ptr() if act else None,
        weight.data_ptr(), res_scale, eps, act, x.numel() // D, D, zr, zs, y.data_ptr(),
        None if h is None else h.data_ptr(), _raw_stream(dev.index))
    if rc != GDN_OK:
        _raise("gdn_norm_gate", rc)
    return y, h


def gdn_norm_gate_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, z: Optional[torch.Tensor] = None,
                      dh: Optional[torch.Tensor] = None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0,
                      workspace: Optional[torch.Tensor] = None):
    """Gradients of gdn_norm_gate: dy, h (what was normed) bf16 [..., D], dh the gradient that reaches h from its other
    uses (None without a residual).  Returns (dx, dresidual, dz, dweight): bf16 but the fp32 dweight [D]; dresidual
    None without dh, dz None without z."""
    dev = h.device
    _need(h, "h", _BF, dev, h.dim())
    _need(dy, "dy", _BF, dev, h.dim())
    D = h.shape[-1] if h.dim() else 0
    _need(weight, "weight", _F32, dev, 1)
    if D < 1 or weight.shape[0] != D or dy.shape != h.shape:
        raise ValueError(f"gdn_norm_gate_bwd: weight must be [{D}], dy of h's shape {tuple(h.shape)}")
    act = _act_of(activation, z, "gdn_norm_gate_bwd")
    zr, zs = _gate_layout(z, h, "gdn_norm_gate_bwd") if act else (0, 0)
    dx = torch.empty_like(h)
    dres = dz = None
    if dh is not None:
        _need(dh, "dh", _BF, dev, h.dim())
        if dh.shape != h.shape:
            raise ValueError("gdn_norm_gate_bwd: dh must have the shape of h")
        dres = torch.empty_like(h)
    if act:
        dz = torch.empty_like(h)
    dw = torch.empty_like(weight)
    lib, rows = load_library(), h.numel() // D
    need = lib.gdn_norm_gate_bwd_workspace_size(rows, D)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, dev, 1)
    rc = lib.gdn_norm_gate_bwd(
        dy.data_ptr(), h.data_ptr(), z.data_ptr() if act else None, None if dh is None else dh.data_ptr(),
        weight.data_ptr(), res_scale, eps, act, rows, D, zr, zs, dx.data_ptr(),
        None if dres is None else dres.data_ptr(), None if dz is None else dz.data_ptr(), dw.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _raw_stream(dev.index))
    if rc != GDN_OK:
        _raise("gdn_norm_gate_bwd", rc)
    return dx, dres, dz, dw


class _NormGate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, z, activation, eps, res_scale):
        y, h = gdn_norm_gate(x, weight, residual=residual, z=z, activation=activation, eps=eps, res_scale=res_scale)
        ctx.save_for_backward(x if h is None else h, weight, z)
        ctx.args = (activation, eps, res_scale, residual is not None)
        return y if h is None else (y, h)

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, z = ctx.saved_tensors
        activation, eps, res_scale, has_res = ctx.args
        if has_res:
            dh = torch.zeros_like(h) if dh is None else dh.to(_BF).contiguous()
        dx, dres, dz, dw = gdn_norm_gate_bwd(dy.to(_BF).contiguous(), h, weight, z=z, dh=dh if has_res else None,
                                             activation=activation, eps=eps, res_scale=res_scale)
        return dx, dw, dres, dz, None, None, None


def norm_gate(x, weight, residual=None, z=None, activation="silu", eps: float = 1e-6, res_scale: float = 1.0):
    """Differentiable gdn_norm_gate: returns (y, h), h None without a residual; gradients for x, weight, residual, z."""
    out = _NormGate.apply(x, weight, residual, z, activation, eps, res_scale)
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
    dev = q.device
    ldq = _rows_dense(q, "q", _BF, dev, 3)
    T, HQ, D = q.shape
    HK = ldk = 0
    if k is not None:
        ldk = _rows_dense(k, "k", _BF, dev, 3)
        HK = k.shape[1]
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"gdn_rope: k must be [{T}, HK, {D}]")
    _need(positions, "positions", _I32, dev, 1)
    _need(inv_freq, "inv_freq", _F32, dev, 1)
    if positions.shape[0] != T:
        raise ValueError("gdn_rope: one position for each token is needed")
    if q_out is None:
        q_out = torch.empty((T, HQ, D), dtype=_BF, device=dev)
    else:
        _need(q_out, "q_out", _BF, dev, 3)
        if q_out.shape != q.shape:
            raise ValueError("gdn_rope: q_out must have the shape of q")
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = torch.empty((T, HK, D), dtype=_BF, device=dev)
    else:
        _need(k_out, "k_out", _BF, dev, 3)
        if k_out.shape != k.shape:
            raise ValueError("gdn_rope: k_out must have the shape of k")
    rc = load_library().gdn_rope(
        q.data_ptr(), None if k is None else k.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), T, HQ, HK, D,
        2 * inv_freq.shape[0], 1 if interleaved else 0, 1 if inverse else 0, attention_factor, ldq, ldk,
        q_out.data_ptr(), None if k is None else k_out.data_ptr(), _raw_stream(dev.index))
    if rc != GDN_OK:
        _raise("gdn_rope", rc)
    return q_out, k_out


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, interleaved, attention_factor):
        ctx.save_for_backward(positions, inv_freq)
        ctx.args = (interleaved, attention_factor)
        return gdn_rope(q, k, positions, inv_freq, interleaved=interleaved, attention_factor=attention_factor)

    @staticmethod
    def backward(ctx, dq, dk):
        positions, inv_freq = ctx.saved_tensors
        interleaved, factor = ctx.args
        dq, dk = gdn_rope(dq.to(_BF).contiguous(), dk.to(_BF).contiguous(), positions, inv_freq, interleaved=interleaved,
                          attention_factor=factor, inverse=True)
        return dq, dk, None, None, None, None


def rotary_embedding(q, k, positions, inv_freq, interleaved: bool = False, attention_factor: float = 1.0):
    """Differentiable gdn_rope of q and k."""
    return _Rotary.apply(q, k, positions, inv_freq, interleaved, attention_factor)


# ------------------------------------------------------------- paged cache
def gdn_paged_plan(cached_lens: torch.Tensor, cu_seqlens: torch.Tensor, block_table: torch.Tensor,
                   free_pages: torch.Tensor, num_free: torch.Tensor, page_size: int, num_tokens: int,
                   dev_status: Optional[torch.Tensor] = None):
    """Pages, slots and positions of one step: see include/gdn.h.  cached_lens int32 [N], cu_seqlens int32 [N + 1],
    block_table int32 [N, width] (entries of new pages written in place), free_pages int32 [F], num_free int32 [1],
    num_tokens = cu_seqlens[N] (a host number, so nothing is read back).  Returns (seq_lens [N], slot_mapping [T],
    positions [T], num_free_out [1]), all int32."""
    dev = cached_lens.device
    _need(cached_lens, "cached_lens", _I32, dev, 1)
    _need(cu_seqlens, "cu_seqlens", _I32, dev, 1)
    _need(block_table, "block_table", _I32, dev, 2)
    _need(free_pages, "free_pages", _I32, dev, 1)
    _need(num_free, "num_free", _I32, dev, 1)
    N, T = cached_lens.shape[0], int(num_tokens)
    if cu_seqlens.shape[0] != N + 1 or block_table.shape[0] != N or num_free.shape[0] != 1:
        raise ValueError("gdn_paged_plan: cu_seqlens [N + 1], block_table [N, width] and num_free [1] must agree")
    if T < 0:
        raise ValueError("gdn_paged_plan: num_tokens must not be negative")
    if dev_status is not None:
        _need(dev_status, "dev_status", _I32, dev, 1)
    # one allocation, the parts on 16-byte boundaries
    n4, t4 = (N + 3) // 4 * 4, (T + 3) // 4 * 4
    buf = torch.empty(n4 + 2 * t4 + 1, dtype=_I32, device=dev)
    seq_lens, slots, pos, left = buf[:N], buf[n4:n4 + T], buf[n4 + t4:n4 + t4 + T], buf[n4 + 2 * t4:]
    at = buf.data_ptr()
    rc = load_library().gdn_paged_plan(
        cached_lens.data_ptr(), cu_seqlens.data_ptr(), N, T, block_table.data_ptr(), block_table.shape[1],
        free_pages.data_ptr(), free_pages.shape[0], num_free.data_ptr(), int(page_size), at, at + 4 * n4,
        at + 4 * (n4 + t4), at + 4 * (n4 + 2 * t4), None if dev_status is None else dev_status.data_ptr(),
        _raw_stream(dev.index))
    if rc != GDN_OK:
        _raise("gdn_paged_plan", rc)
    return seq_lens, slots, pos, left


def _cache_args(k_cache, v_cache, k_scale, v_scale, dev, fn):
    _need(k_cache, "k_cache", _F8, dev, 4)
    _need(v_cache, "v_cache", _F8, dev, 4)
    _need(k_scale, "k_scale", _F32, dev, 2)
    _need(v_scale, "v_scale", _F32, dev, 2)
    shape = k_cache.shape
    if v_cache.shape != shape or k_scale.shape != shape[:2] or v_scale.shape != shape[:2]:
        raise ValueError(f"{fn}: caches must be [P, HK, page_size, D] and scales [P, HK]")
    return shape


def gdn_kv8_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   k_scale: torch.Tensor, v_scale: torch.Tensor, slot_mapping: torch.Tensor,
                   dev_status: Optional[torch.Tensor] = None) -> None:
    """New keys and values into the 8-bit cache, in place.  k, v bf16 [T, HK, D] (any token stride); k_cache, v_cache
    float8_e4m3fn [P, HK, page_size, D]; k_scale, v_scale fp32 [P, HK]; slot_mapping int32 [T] (-1 skips a token)."""
    dev = k.device
    ldk, ldv = _rows_dense(k, "k", _BF, dev, 3), _rows_dense(v, "v", _BF, dev, 3)
    P, HK, bs, D = _cache_args(k_cache, v_cache, k_scale, v_scale, dev, "gdn_kv8_append")
    _need(slot_mapping, "slot_mapping", _I32, dev, 1)
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1] != HK or k.shape[2] != D or slot_mapping.shape[0] != T:
        raise ValueError(f"gdn_kv8_append: k, v must be [T, {HK}, {D}] and slot_mapping [T]")
    if dev_status is not None:
        _need(dev_status, "dev_status", _I32, dev, 1)
    rc = load_library().gdn_kv8_append(
        k.data_ptr(), v.data_ptr(), ldk, ldv, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), slot_mapping.data_ptr(), T, P, HK, D, bs,
        None if dev_status is None else dev_status.data_ptr(), _raw_stream(dev.index))
    if rc != GDN_OK:
        _raise("gdn_kv8_append", rc)


def kv8_attention_workspace_size(N, T, HQ, HK, D, max_q_len, max_seq_len) -> int:
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
    dev = q.device
    ldq = _rows_dense(q, "q", _BF, dev, 3)
    T, HQ, D = q.shape
    P, HK, bs, Dc = _cache_args(k_cache, v_cache, k_scale, v_scale, dev, "gdn_kv8_attention")
    _need(block_table, "block_table", _I32, dev, 2)
    _need(seq_lens, "seq_lens", _I32, dev, 1)
    N, width = block_table.shape
    if Dc != D or seq_lens.shape[0] != N:
        raise ValueError("gdn_kv8_attention: q and the caches must agree in D, block_table and seq_lens in N")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", _I32, dev, 1)
        if cu_seqlens.shape[0] != N + 1:
            raise ValueError("gdn_kv8_attention: cu_seqlens must be [N + 1]")
    if max_seq_len is None:
        max_seq_len = width * bs
    if o is None:
        o = torch.empty((T, HQ, D), dtype=_BF, device=dev)
    else:
        _need(o, "o", _BF, dev, 3)
        if o.shape != q.shape:
            raise ValueError("gdn_kv8_attention: o must have the shape of q")
    if lse is not None:
        _need(lse, "lse", _F32, dev, 2)
        if lse.shape != q.shape[:2]:
            raise ValueError("gdn_kv8_attention: lse must be [T, HQ]")
    if dev_status is not None:
        _need(dev_status, "dev_status", _I32, dev, 1)
    lib = load_library()
    if workspace is None:
        need = lib.gdn_kv8_attention_workspace_size(N, T, HQ, HK, D, max_q_len, max_seq_len)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, dev, 1)
    rc = lib.gdn_kv8_attention(
        q.data_ptr(), ldq, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), width, seq_lens.data_ptr(), None if cu_seqlens is None else cu_seqlens.data_ptr(), N, T, P,
        HQ, HK, D, bs, int(max_q_len), int(max_seq_len), -1.0 if scale is None else scale, o.data_ptr(),
        None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), None if dev_status is None else dev_status.data_ptr(),
        _raw_stream(dev.index))
    if rc != GDN_OK:
        _raise("gdn_kv8_attention", rc)
    return o
