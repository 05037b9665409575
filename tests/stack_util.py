"""Plain 64-bit implementations (NumPy, one loop a definition) of the operators around the recurrence, written from
include/gdn.h and independent of the library."""
import math

import numpy as np
import torch

EXP_MIN = -60


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def bf16(x):
    """Round a float64 array to bf16 (torch, to nearest even) and back."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16)


def act(z, kind):
    s = 1.0 / (1.0 + np.exp(-z))
    if kind == "silu":
        return z * s, s * (1.0 + z * (1.0 - s))
    return s, s * (1.0 - s)


def norm_fwd(x, w, res=None, z=None, kind="silu", eps=1e-6, res_scale=1.0):
    h = x if res is None else res + res_scale * x
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w
    if z is not None:
        y = y * act(z, kind)[0]
    return y, h


def norm_bwd(dy, h, w, z=None, dh=None, kind="silu", eps=1e-6, res_scale=1.0):
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n = h * r
    f, d = (np.ones_like(h), None) if z is None else act(z, kind)
    u = dy * f
    p = u * w
    dH = r * (p - n * (p * n).mean(-1, keepdims=True)) + (0.0 if dh is None else dh)
    dz = None if z is None else dy * n * w * d
    return res_scale * dH, dH, dz, (u * n).reshape(-1, h.shape[-1]).sum(0)


def rope(x, pos, inv_freq, interleaved, factor=1.0, inverse=False):
    """x [T, H, D] float64, inv_freq the fp32 values; the angle is exact (Python integers and long double are not
    needed: position x inv_freq has at most 31 + 24 bits, and float64 keeps 53 of them)."""
    rot = 2 * len(inv_freq)
    ang = pos.astype(np.float64)[:, None] * inv_freq.astype(np.float64)[None, :]
    c, s = np.cos(ang)[:, None] * factor, np.sin(ang)[:, None] * factor * (-1.0 if inverse else 1.0)
    y = x.copy()
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def plan(cached, cu, table, free, left, bs, T):
    """Lists in, lists out; returns (table, seq_lens, slots, positions, left, a page was missing)."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    slots, pos, lens, missing = [-1] * T, [0] * T, [], False
    for n, c in enumerate(cached):
        new = cu[n + 1] - cu[n]
        lens.append(c + new)
        have, need = -(-c // bs), -(-(c + new) // bs)
        for p in range(have, need):
            if p >= width:
                missing = True
                break
            if left > 0:
                left -= 1
                table[n][p] = free[left]
            else:
                table[n][p] = -1
                missing = True
        for i in range(new):
            at = c + i
            pos[cu[n] + i] = at
            page = table[n][at // bs] if at // bs < width else -1
            slots[cu[n] + i] = page * bs + at % bs if page >= 0 else -1
    return table, lens, slots, pos, left, missing


def to_e4m3(x):
    """Values of the 8-bit format nearest to x (ties to even), infinities to +-448; NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        y = np.clip(x, -448.0, 448.0)
        e = np.frexp(np.where(np.isnan(y), 1.0, y))[1]
        step = np.ldexp(1.0, np.maximum(e, -5) - 4)
        out = np.round(y / step) * step  # numpy rounds halves to even
        return np.clip(out, -448.0, 448.0)


def least_exponent(amax):
    e = EXP_MIN
    if amax > 0:
        m, x = math.frexp(amax)
        e = max(EXP_MIN, x - 9 + (1 if m > 0.875 else 0))
    return e


def append(x, codes, scale, slots):
    """x [T, H, D], codes [P, H, bs, D] (values), scale [P, H]; returns new (codes, scale)."""
    codes, scale = codes.copy(), scale.copy()
    P, H, bs, _ = codes.shape
    t = 0
    while t < len(slots):
        s = slots[t]
        if s < 0 or s >= P * bs:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % bs:
            n += 1
        pg, off = s // bs, s % bs
        for h in range(H):
            new = x[t:t + n, h]
            fin = np.abs(new[np.isfinite(new)])
            e = least_exponent(float(fin.max()) if fin.size else 0.0)
            if off:
                old = int(round(math.log2(scale[pg, h])))
                e = max(e, old)
                if e > old:
                    codes[pg, h, :off] = to_e4m3(codes[pg, h, :off] * 2.0 ** (old - e))
            codes[pg, h, off:off + n] = to_e4m3(new * 2.0 ** -e)
            scale[pg, h] = 2.0 ** e
        t += n
    return codes, scale


def attention(q, kc, vc, ks, vs, table, lens, cu, scale):
    """q [T, HQ, D] float64; kc, vc code values [P, HK, bs, D]; returns o, lse and sum_j p_ij |v_j| (for bounds)."""
    T, HQ, D = q.shape
    P, HK, bs, _ = kc.shape
    G = HQ // HK
    o, mag = np.zeros((T, HQ, D)), np.zeros((T, HQ, D))
    lse = np.full((T, HQ), -np.inf)
    for n, L in enumerate(lens):
        m = cu[n + 1] - cu[n]
        if m == 0:
            continue
        pages = [table[n][p] for p in range(-(-L // bs))]
        for hk in range(HK):
            if L:
                K = np.concatenate([kc[p, hk] * ks[p, hk] if 0 <= p < P else np.zeros((bs, D)) for p in pages])[:L]
                V = np.concatenate([vc[p, hk] * vs[p, hk] if 0 <= p < P else np.zeros((bs, D)) for p in pages])[:L]
                there = np.repeat([0 <= p < P for p in pages], bs)[:L]
            for i in range(m):
                seen = max(0, L - m + i + 1)
                if seen == 0 or not there[:seen].any():
                    continue
                for g in range(G):
                    hq = hk * G + g
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = np.where(there[:seen], K[:seen] @ q[cu[n] + i, hq] * scale, -np.inf)
                        top = s.max()
                        p = np.exp(s - top)
                        l = p.sum()
                        o[cu[n] + i, hq] = (p @ np.where(there[:seen, None], V[:seen], 0.0)) / l
                        mag[cu[n] + i, hq] = (p @ np.abs(np.where(there[:seen, None], V[:seen], 0.0))) / l
                        lse[cu[n] + i, hq] = top + np.log(l)
    return o, lse, mag


def make_cache(P, HK, bs, D, gen, spread=0.5):
    """Random codes and power-of-two scales: (codes float8 [P, HK, bs, D], scale fp32 [P, HK]) on the CPU."""
    x = torch.randn(P, HK, bs, D, generator=gen) * torch.exp(spread * torch.randn(P, HK, 1, 1, generator=gen))
    e = torch.tensor([[least_exponent(float(x[p, h].abs().max())) for h in range(HK)] for p in range(P)])
    sc = torch.ldexp(torch.ones(P, HK), e)
    return (x / sc[:, :, None, None]).to(torch.float8_e4m3fn), sc
