"""Cases of the operators of a training step through a stack of gated-delta-rule and attention layers.

Three operators, each direction in its plain form (elementary torch operations in 32 bits) and through the package's
entry points:

* ``attn``   attention of packed sequences (``gdn_attention_fwd``) and its gradient, which forms the probabilities again
             from the logsumexp (``gdn_attention_bwd``)
* ``act8``   activations kept for the backward pass as 8-bit codes, one power-of-two scale for each 128 elements of a
             row (``gdn_act8_save``, ``gdn_act8_load``)
* ``norm8``  RMS norm with a gate and a scaled residual whose forward writes such codes of what its backward needs
             (``gdn_norm_gate_save8``), and the backward from them (``gdn_norm_gate_bwd8``)

Sequence lengths are a fixed spread over [lo, hi] in an order drawn from the seed, so that the work of a case does not
depend on the seed.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
EXP_MIN = -60  # lowest exponent of a scale
GROUP = 128    # elements of a row that share a scale
AT_ONCE = 1 << 28  # logits that the plain form holds at once


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the attention layer of a small training step: one sequence, a few heads, latency
        {"name": "attn_step_fwd", "op": "attn", "dir": "fwd", "seqs": 1, "lo": 256, "hi": 256, "more_keys": 0, "causal": True,
         "hq": 8, "hkv": 2, "dim": 128},
        # a packed batch of ragged documents
        {"name": "attn_packed_fwd", "op": "attn", "dir": "fwd", "seqs": 24, "lo": 200, "hi": 2000, "more_keys": 0, "causal": True,
         "hq": 32, "hkv": 4, "dim": 128},
        # one long document
        {"name": "attn_long_fwd", "op": "attn", "dir": "fwd", "seqs": 1, "lo": 16384, "hi": 16384, "more_keys": 0, "causal": True,
         "hq": 32, "hkv": 4, "dim": 128},
        # the gradients of the same three (the long one half as long: a training step of 8192 tokens)
        {"name": "attn_step_bwd", "op": "attn", "dir": "bwd", "seqs": 1, "lo": 256, "hi": 256, "more_keys": 0, "causal": True,
         "hq": 8, "hkv": 2, "dim": 128},
        {"name": "attn_packed_bwd", "op": "attn", "dir": "bwd", "seqs": 24, "lo": 200, "hi": 2000, "more_keys": 0, "causal": True,
         "hq": 32, "hkv": 4, "dim": 128},
        {"name": "attn_long_bwd", "op": "attn", "dir": "bwd", "seqs": 1, "lo": 8192, "hi": 8192, "more_keys": 0, "causal": True,
         "hq": 32, "hkv": 4, "dim": 128},
        # attention without a mask over keys of another length, small heads, no groups
        {"name": "attn_cross_bwd", "op": "attn", "dir": "bwd", "seqs": 6, "lo": 300, "hi": 1500, "more_keys": 777, "causal": False,
         "hq": 16, "hkv": 16, "dim": 64},
        # what the projections of a step of 8192 tokens keep: one input of the model's width, a slice of a wider tensor
        {"name": "act8_save_train", "op": "act8", "dir": "save", "tokens": 8192, "dim": 4096, "packed": True},
        # and its return for the weight's gradient in the small training step
        {"name": "act8_load_step", "op": "act8", "dir": "load", "tokens": 256, "dim": 512, "packed": False},
        # the gated norm after the recurrence in a step of 2 x 4096 tokens, 32 value heads, with its codes
        {"name": "norm8_gate_train_fwd", "op": "norm8", "dir": "fwd", "tokens": 8192, "heads": 32, "dim": 128, "act": "silu",
         "residual": False},
        # its gradient from the codes
        {"name": "norm8_gate_train_bwd", "op": "norm8", "dir": "bwd", "tokens": 8192, "heads": 32, "dim": 128, "act": "silu",
         "residual": False},
        # the gradient of a norm before a block: one token a row, the residual stream's gradient joins
        {"name": "norm8_stream_bwd", "op": "norm8", "dir": "bwd", "tokens": 4001, "heads": 1, "dim": 4096, "act": "none",
         "residual": True},
    ]


def _log(rng, lo, hi):
    """A whole number, spread over its logarithm, odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "act8", "norm8"])
    if op == "attn":
        way = rng.choice(["fwd", "bwd"])
        hkv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8]), rng.choice([64, 128])
        causal = rng.random() < 0.8
        most = (8192 * 8192 // 2) * 32 * 128 // (hkv * group * dim)  # (row, key) pairs of a head, of all sequences
        seqs = min(_log(rng, 1, 48), max(1, most // 64))
        hi = _log(rng, 1, max(1, min(16384, int(math.sqrt(most / seqs)))))
        # keys before the sequence's own (kept from an earlier segment, or another tensor's), or fewer keys than rows
        more = rng.choice([0, 0, 0, _log(rng, 1, max(1, hi // 2)), -_log(rng, 1, max(1, hi // 2))])
        return {"op": "attn", "dir": way, "seqs": seqs, "lo": max(1, hi // rng.choice([1, 2, 8])), "hi": hi, "more_keys": more,
                "causal": causal, "hq": hkv * group, "hkv": hkv, "dim": dim}
    if op == "act8":
        dim = rng.choice([64, 96, 128, 512, 1000, 2048, 4096, 5120, 8192])
        return {"op": "act8", "dir": rng.choice(["save", "load"]), "tokens": _log(rng, 1, max(1, 8192 * 4096 // dim)), "dim": dim,
                "packed": rng.random() < 0.5}
    if rng.random() < 0.5:  # the norm after a block, one head a row
        heads, dim = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 96, 128, 256])
    else:  # the norm before a block, one token a row
        heads, dim = 1, rng.choice([512, 1000, 2048, 4096, 5120, 8192])
    tokens = _log(rng, 1, max(1, (8192 * 32 * 128) // (heads * dim * 2)))
    return {"op": "norm8", "dir": rng.choice(["fwd", "bwd"]), "tokens": tokens, "heads": heads, "dim": dim,
            "act": rng.choice(["none", "silu", "sigmoid"]), "residual": rng.random() < 0.5}


def _spread(lo, hi, count):
    """`count` whole numbers over [lo, hi], the same for every seed; the first is hi."""
    return [hi - int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0) * 0.999999) for i in range(count)]


def _lengths(case):
    """(rows, keys) of each sequence."""
    rows = _spread(case["lo"], case["hi"], case["seqs"])
    return rows, [max(0, m + case["more_keys"]) for m in rows]


# --------------------------------------------------------------- 8-bit codes
def _exponents(amax):
    """The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8 is the largest value of the 8-bit format), at least EXP_MIN."""
    mant, exp = torch.frexp(amax)  # amax = mant * 2^exp, mant in [0.5, 1)
    e = exp - 9 + (mant > 0.875).to(exp.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(min=EXP_MIN)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _encode(x):
    """bf16 [..., D] -> (codes e4m3 [..., D], scales fp32 [..., ceil(D / GROUP)])."""
    D = x.shape[-1]
    groups = -(-D // GROUP)
    x = torch.nn.functional.pad(x.float(), (0, groups * GROUP - D)).unflatten(-1, (groups, GROUP))
    e = _exponents(x.abs().amax(-1))
    codes = (x * _pow2(-e)[..., None]).to(F8)
    return codes.flatten(-2)[..., :D].contiguous(), _pow2(e)


def _decode(codes, scale):
    """The fp32 values that codes and scales stand for."""
    return codes.float() * scale.repeat_interleave(GROUP, -1)[..., :codes.shape[-1]]


# ----------------------------------------------------------------- prepare
def prepare(case, seed):
    dev, bf = "cuda", torch.bfloat16
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    r = random.Random(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case)
    op, D = case["op"], case["dim"]
    if op == "attn":
        pairs = list(zip(*_lengths(case)))
        r.shuffle(pairs)
        s["spans"], tq, tk = [], 0, 0  # (first row, rows, first key, keys)
        for m, n in pairs:
            s["spans"].append((tq, m, tk, n))
            tq, tk = tq + m, tk + n
        s["cu"] = torch.tensor([a for a, _, _, _ in s["spans"]] + [tq], dtype=torch.int32, device=dev)
        s["cu_k"] = None
        hq, hkv = case["hq"], case["hkv"]
        if case["more_keys"] == 0:  # as they leave a packed projection: views with a longer token stride
            qkv = randn(tq, (hq + 2 * hkv) * D).to(bf)
            s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in qkv.split([hq * D, hkv * D, hkv * D], dim=1))
        else:
            s["cu_k"] = torch.tensor([a for _, _, a, _ in s["spans"]] + [tk], dtype=torch.int32, device=dev)
            kv = randn(tk, 2 * hkv * D).to(bf)
            s["q"] = randn(tq, hq, D).to(bf)
            s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in kv.split(hkv * D, dim=1))
        s["q"].mul_(2.0)  # logits of a standard deviation of 2
        s["scale"] = D ** -0.5
        if case["dir"] == "bwd":
            s["o"], s["lse"] = _plain_attn_fwd(s)
            s["do"] = randn(tq, hq, D).to(bf)
        return s
    if op == "act8":
        x = (randn(case["tokens"], D) * torch.exp(0.5 * randn(1, D)) * torch.exp(0.25 * randn(case["tokens"], 1))).to(bf)
        if case["dir"] == "load":
            s["codes"], s["scales"] = _encode(x)
        elif case["packed"]:  # a slice of a wider tensor
            wide = torch.zeros(case["tokens"], D + 1024, dtype=bf, device=dev)
            s["x"] = wide[:, 512:512 + D]
            s["x"].copy_(x)
        else:
            s["x"] = x
        return s
    T, H = case["tokens"], case["heads"]
    shape = (T, H, D) if H > 1 else (T, D)
    x = (2.0 * randn(*shape)).to(bf)
    z = randn(*shape).to(bf) if case["act"] != "none" else None
    s["weight"] = 1.0 + 0.1 * randn(D)
    s["res_scale"] = 0.5 if case["residual"] else 1.0
    s["eps"] = 1e-6
    if case["dir"] == "fwd":
        s["x"], s["z"] = x, z
        s["res"] = (2.0 * randn(*shape)).to(bf) if case["residual"] else None
    else:
        s["h8"] = _encode(x)
        s["z8"] = _encode(z) if z is not None else (None, None)
        s["dy"] = randn(*shape).to(bf)
        s["dh"] = randn(*shape).to(bf) if case["residual"] else None
    return s


# --------------------------------------------------------------------- run
def run(s):
    return (_own if own else _plain)[s["op"], s["dir"]](s)


def _own_attn_fwd(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn.gdn_attention_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"], causal=s["causal"],
                                 scale=s["scale"])


def _own_attn_bwd(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn.gdn_attention_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"],
                                 causal=s["causal"], scale=s["scale"])


def _own_act8_save(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn.gdn_act8_save(s["x"])


def _own_act8_load(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn.gdn_act8_load(s["codes"], s["scales"])


def _own_norm8_fwd(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    act = None if s["act"] == "none" else s["act"]
    return gdn.gdn_norm_gate_save8(s["x"], s["weight"], residual=s["res"], z=s["z"], activation=act, eps=s["eps"],
                                   res_scale=s["res_scale"])


def _own_norm8_bwd(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    act = None if s["act"] == "none" else s["act"]
    return gdn.gdn_norm_gate_bwd8(s["dy"], *s["h8"], s["weight"], *s["z8"], dh=s["dh"], activation=act, eps=s["eps"],
                                  res_scale=s["res_scale"])


def _blocks(s):
    """(rows, keys, kv head, query heads) of one sequence at a time, as many query heads of a kv head at once as fit."""
    group = s["hq"] // s["hkv"]
    for a, m, b, n in s["spans"]:
        step = max(1, min(group, AT_ONCE // max(1, m * n)))
        for h in range(s["hkv"]):
            for g in range(0, group, step):
                yield slice(a, a + m), slice(b, b + n), h, slice(h * group + g, h * group + min(g + step, group))


def _masked(logits, causal):
    """Row i of m sees the keys up to i + n - m of n."""
    m, n = logits.shape[-2:]
    if causal:
        seen = torch.arange(n, device=logits.device) <= torch.arange(m, device=logits.device)[:, None] + (n - m)
        logits.masked_fill_(~seen, -math.inf)
    return logits


def _plain_attn_fwd(s):
    q, k, v = s["q"], s["k"], s["v"]
    o = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device)
    for rows, keys, h, heads in _blocks(s):
        if keys.start == keys.stop:
            continue
        p = torch.matmul(q[rows, heads].float().transpose(0, 1), k[keys, h].float().T).mul_(s["scale"])
        _masked(p, s["causal"])
        top = p.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        got = torch.matmul(p, v[keys, h].float()) / torch.where(total == 0, torch.ones_like(total), total)
        o[rows, heads] = got.transpose(0, 1).to(torch.bfloat16)
        lse[rows, heads] = (top + torch.log(total))[..., 0].T
    return o, lse


def _plain_attn_bwd(s):
    q, k, v, do, scale = s["q"], s["k"], s["v"], s["do"], s["scale"]
    dq = torch.zeros(q.shape, device=q.device)
    dk, dv = torch.zeros(k.shape, device=q.device), torch.zeros(v.shape, device=q.device)
    delta = (do.float() * s["o"].float()).sum(-1)
    for rows, keys, h, heads in _blocks(s):
        if keys.start == keys.stop:
            continue
        qf, kf, vf, df = (t.float() for t in (q[rows, heads].transpose(0, 1), k[keys, h], v[keys, h], do[rows, heads].transpose(0, 1)))
        p = _masked(torch.matmul(qf, kf.T).mul_(scale), s["causal"])
        lse = s["lse"][rows, heads].T[..., None]
        p.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
        dv[keys, h] += torch.matmul(p.transpose(1, 2), df).sum(0)
        p.mul_(torch.matmul(df, vf.T).sub_(delta[rows, heads].T[..., None]))
        dq[rows, heads] = torch.matmul(p, kf).mul_(scale).transpose(0, 1)
        dk[keys, h] += torch.matmul(p.transpose(1, 2), qf).sum(0).mul_(scale)
    return dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _plain_act8_save(s):
    return _encode(s["x"])


def _plain_act8_load(s):
    return _decode(s["codes"], s["scales"]).to(torch.bfloat16)


def _plain_norm8_fwd(s):
    x = s["x"].float()
    h = x if s["res"] is None else s["res"].float() + s["res_scale"] * x
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    z8 = (None, None)
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        y = y * (sig if s["act"] == "sigmoid" else z * sig)
        z8 = _encode(s["z"])
    kept = h.to(torch.bfloat16)
    return (y.to(torch.bfloat16), None if s["res"] is None else kept) + _encode(kept) + z8


def _plain_norm8_bwd(s):
    h, w, dy = _decode(*s["h8"]), s["weight"], s["dy"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"])
    n = h * rstd
    gate, dz = 1.0, None
    if s["z8"][0] is not None:
        z = _decode(*s["z8"])
        sig = 1.0 / (1.0 + torch.exp(-z))
        gate = sig if s["act"] == "sigmoid" else z * sig
        slope = sig * (1.0 - sig) if s["act"] == "sigmoid" else sig * (1.0 + z * (1.0 - sig))
        dz = (dy * n * w * slope).to(torch.bfloat16)
    u = dy * gate
    p = u * w
    dh = rstd * (p - n * (p * n).mean(-1, keepdim=True))
    dres = None
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
        dres = dh.to(torch.bfloat16)
    return (s["res_scale"] * dh).to(torch.bfloat16), dres, dz, (u * n).reshape(-1, n.shape[-1]).sum(0)


_own = {("attn", "fwd"): _own_attn_fwd, ("attn", "bwd"): _own_attn_bwd, ("act8", "save"): _own_act8_save,
        ("act8", "load"): _own_act8_load, ("norm8", "fwd"): _own_norm8_fwd, ("norm8", "bwd"): _own_norm8_bwd}
_plain = {("attn", "fwd"): _plain_attn_fwd, ("attn", "bwd"): _plain_attn_bwd, ("act8", "save"): _plain_act8_save,
          ("act8", "load"): _plain_act8_load, ("norm8", "fwd"): _plain_norm8_fwd, ("norm8", "bwd"): _plain_norm8_bwd}


# -------------------------------------------------------------------- work
def work(case):
    op, D = case["op"], case["dim"]
    if op == "attn":
        rows, keys = _lengths(case)
        pairs = 0
        for m, n in zip(rows, keys):
            if not case["causal"]:
                pairs += m * n
            else:  # row i sees max(0, n - m + i + 1) keys
                t = min(m, n)
                pairs += t * (n - t) + t * (t + 1) // 2
        q, kv, bwd = sum(rows) * case["hq"], sum(keys) * case["hkv"], case["dir"] == "bwd"
        # q, k, v in and o, lse out; or q, o, do, lse, k, v in and dq, dk, dv out
        return {"bytes": 2 * D * (4 * q + 4 * kv) + 4 * q if bwd else 2 * D * (2 * q + 2 * kv) + 4 * q,
                "flops": (10 if bwd else 4) * pairs * case["hq"] * D}
    groups = -(-D // GROUP)
    if op == "act8":
        return {"bytes": case["tokens"] * (3 * D + 4 * groups), "flops": 2 * case["tokens"] * D}
    rows, gate, res = case["tokens"] * case["heads"], case["act"] != "none", case["residual"]
    if case["dir"] == "fwd":  # x, y; residual, h; z; codes and scales of h and of z
        each = D * (4 + 4 * res + 2 * gate) + (D + 4 * groups) * (1 + gate)
        return {"bytes": rows * each + 4 * D, "flops": 10 * rows * D}
    # dy, dx; dh, dresidual; dz; codes and scales
    each = D * (4 + 4 * res + 2 * gate) + (D + 4 * groups) * (1 + gate)
    return {"bytes": rows * each + 8 * D, "flops": 10 * rows * D}


# ------------------------------------------------------------------- exact
def _to8(x):
    """x rounded to the 8-bit format's values: three bits after the leading one, steps of 2^-9 below 2^-6, ties to even."""
    exp = torch.frexp(x)[1].clamp(min=-5)
    step = ((exp.long() - 4 + 1023) << 52).view(torch.float64)  # 2^(exp - 4) from its bits: a power on the GPU may be off by one
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits."""
    f = torch.float64

    def codes(x):  # group by group
        parts, scales = [], []
        for x in x.to(f).split(GROUP, -1):
            amax = x.abs().amax(-1, keepdim=True)
            scale = torch.full_like(amax, 2.0 ** EXP_MIN)  # doubled until the largest magnitude fits: exact in 64 bits
            while bool((amax > 448.0 * scale).any()):
                scale = torch.where(amax > 448.0 * scale, 2.0 * scale, scale)
            scales.append(scale)
            parts.append(_to8(x / scale))
        return torch.cat(parts, -1), torch.cat(scales, -1)

    def values(c, scale):
        return torch.cat([part.to(f) * scale[..., i:i + 1].to(f) for i, part in enumerate(c.view(torch.uint8).split(GROUP, -1))
                          for part in [part.view(F8)]], -1)

    def attn(s):
        q, k, v, D = s["q"], s["k"], s["v"], s["dim"]
        G, bwd = s["hq"] // s["hkv"], s["dir"] == "bwd"
        new = lambda t: torch.zeros(t.shape, dtype=f, device=t.device)  # noqa: E731
        o, lse = new(q), torch.full(q.shape[:2], -math.inf, dtype=f, device=q.device)
        dq, dk, dv = new(q), new(k), new(v)
        for a, m, b, n in s["spans"]:
            if n == 0:
                continue
            for h in range(s["hkv"]):
                kk, vv = k[b:b + n, h].to(f), v[b:b + n, h].to(f)
                for hq in range(h * G, h * G + G):
                    for i in range(0, m, 1024):  # rows at once, and the keys that they see
                        count = min(1024, m - i)
                        upto = min(n, n - m + i + count) if s["causal"] else n
                        if upto <= 0:
                            continue
                        at = slice(a + i, a + i + count)
                        qq, kt, vt = q[at, hq].to(f), kk[:upto], vv[:upto]
                        w = torch.einsum("td,kd->tk", qq, kt) * s["scale"]
                        if s["causal"]:
                            hidden = torch.ones(count, upto, dtype=torch.bool, device=w.device).triu(n - m + i + 1)
                            w = w.masked_fill(hidden, -math.inf)
                        if not bwd:
                            lse[at, hq] = torch.logsumexp(w, -1)
                            o[at, hq] = torch.softmax(w, -1).nan_to_num(0.0) @ vt
                            continue
                        p = torch.exp(w - s["lse"][at, hq, None].to(f).clamp(min=-1e300))
                        d = s["do"][at, hq].to(f)
                        dv[b:b + upto, h].addmm_(p.T, d)
                        inner = torch.einsum("td,td->t", d, s["o"][at, hq].to(f))
                        ds = (d @ vt.T - inner[:, None]) * p * s["scale"]
                        dq[at, hq] = ds @ kt
                        dk[b:b + upto, h].addmm_(ds.T, qq)
        return (dq, dk, dv) if bwd else (o, lse)

    def act8(s):
        return codes(s["x"]) if s["dir"] == "save" else values(s["codes"], s["scales"])

    def norm8(s):
        w = s["weight"].to(f)
        bwd = s["dir"] == "bwd"
        gated = s["act"] != "none"
        z = None if not gated else values(*s["z8"]) if bwd else s["z"].to(f)
        sig = torch.sigmoid(z) if gated else None
        gate = 1.0 if not gated else sig if s["act"] == "sigmoid" else sig * z
        if not bwd:
            h = s["x"].to(f) if s["res"] is None else torch.add(s["res"].to(f), s["x"].to(f), alpha=s["res_scale"])
            y = h * h.square().mean(-1, keepdim=True).add(s["eps"]).rsqrt() * (w * gate)
            kept = s["x"] if s["res"] is None else h.to(torch.bfloat16)  # the codes are those of the stored stream
            return (y, None if s["res"] is None else h) + codes(kept) + (codes(s["z"]) if gated else (None, None))
        x, dy = values(*s["h8"]), s["dy"].to(f)
        D = x.shape[-1]
        inv = x.square().mean(-1, keepdim=True).add(s["eps"]).rsqrt()
        up = dy * gate * w
        dh = up * inv - x * ((up * x).sum(-1, keepdim=True) * inv ** 3 / D)
        if s["dh"] is not None:
            dh = dh + s["dh"].to(f)
        dz = None
        if gated:
            d = sig * (1 - sig)
            dz = dy * w * (x * inv) * (d if s["act"] == "sigmoid" else sig + z * d)
        dw = torch.einsum("rd,rd->d", (dy * gate).reshape(-1, D), (x * inv).reshape(-1, D))
        return s["res_scale"] * dh, dh if s["dh"] is not None else None, dz, dw

    return {"attn": attn, "act8": act8, "norm8": norm8}[case["op"]](prepare(case, seed))
