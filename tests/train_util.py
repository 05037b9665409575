"""Plain 64-bit implementations of a training step's operators, written from include/gdn.h and independent of the library,
with the magnitudes that the tests' tolerances are made of."""
import math

import torch

F = torch.float64


def spans(lens, lens_k=None):
    """(first row, rows, first key, keys) of each sequence."""
    out, a, b = [], 0, 0
    for m, n in zip(lens, lens if lens_k is None else lens_k):
        out.append((a, m, b, n))
        a, b = a + m, b + n
    return out


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)


def attention(q, k, v, spans, causal, scale, do=None):
    """Values and, with do, gradients; beside each result what bounds its roundings.  Tensors of any type, on one device.

    Returns a dict: o, o_mag = sum p |v|, lse, lse_mag = 1 + the largest scale sum |q| |k| that is seen;
    dq, dk, dv and for each of them *_round = the sum of the magnitudes of the terms that are rounded to bf16 on their
    way, *_fp32 = the sum of magnitudes that enter in fp32 only, *_delta = that of delta's terms."""
    q, k, v = q.to(F), k.to(F), v.to(F)
    Tq, HQ, D = q.shape
    Tk, HK, _ = k.shape
    G = HQ // HK
    f = dict(dtype=F, device=q.device)
    r = dict(o=torch.zeros_like(q), o_mag=torch.zeros_like(q), lse=torch.full((Tq, HQ), -math.inf, **f), lse_mag=torch.ones(Tq, HQ, **f))
    if do is not None:
        do = do.to(F)
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            for x in ("", "_round", "_fp32", "_delta"):
                r[n + x] = torch.zeros_like(t)
    for a, m, b, n in spans:
        if m == 0 or n == 0:
            continue
        rows, keys = slice(a, a + m), slice(b, b + n)
        seen = torch.ones(m, n, dtype=torch.bool, device=q.device)
        if causal:
            seen = seen.tril(n - m)
        for h in range(HQ):
            K, V, Q = k[keys, h // G], v[keys, h // G], q[rows, h]
            s = (Q @ K.T * scale).masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
            o = p @ V
            r["o"][rows, h], r["o_mag"][rows, h], r["lse"][rows, h] = o, p @ V.abs(), lse
            r["lse_mag"][rows, h] += ((Q.abs() @ K.abs().T) * scale * seen).amax(-1)
            if do is None:
                continue
            d = do[rows, h]
            ds = p * (d @ V.T - (d * o).sum(-1, keepdim=True))
            mag = p * (d.abs() @ V.abs().T + (d * o).abs().sum(-1, keepdim=True)) * r["lse_mag"][rows, h][:, None]
            r["dq"][rows, h] = scale * ds @ K
            r["dq_round"][rows, h] = scale * ds.abs() @ K.abs()
            r["dq_fp32"][rows, h] = scale * mag @ K.abs()
            delta = p * (d * o).abs().sum(-1, keepdim=True)
            r["dq_delta"][rows, h] = scale * delta @ K.abs()
            r["dk_delta"][keys, h // G] += scale * delta.T @ Q.abs()
            r["dk"][keys, h // G] += scale * ds.T @ Q
            r["dk_round"][keys, h // G] += scale * ds.abs().T @ Q.abs()
            r["dk_fp32"][keys, h // G] += scale * mag.T @ Q.abs()
            r["dv"][keys, h // G] += p.T @ d
            r["dv_round"][keys, h // G] += p.T @ d.abs()
            r["dv_fp32"][keys, h // G] += (p * r["lse_mag"][rows, h][:, None]).T @ d.abs()
    return r
