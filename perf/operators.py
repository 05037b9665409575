"""Cases of the operators that stand around the recurrence in a stack of gated-delta-rule and attention layers.

Five operators, each in its plain form (elementary torch operations in 32 bits) and through the package's entry points:

* ``norm``    RMS norm with a gate and a scaled residual (``gdn_norm_gate``, ``gdn_norm_gate_bwd``)
* ``rope``    rotary positions (``gdn_rope``; the backward is the inverse rotation)
* ``plan``    block tables, slot maps and positions from request lengths (``gdn_paged_plan``)
* ``append``  new keys and values into an 8-bit cache, one power-of-two scale for each page and head (``gdn_kv8_append``)
* ``attn``    attention over that cache (``gdn_kv8_attention``)

Request lengths are a fixed spread over [lo, hi] in an order drawn from the seed, so that the work of a case does not
depend on the seed.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
EXP_MIN = -60  # lowest exponent of a page's scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the gated norm after one decode step of 256 requests, 32 value heads: a few microseconds of memory traffic
        {"name": "norm_gate_decode", "op": "norm", "dir": "fwd", "tokens": 256, "heads": 32, "dim": 128, "act": "silu",
         "residual": False},
        # its gradient in a training step of 2 x 4096 tokens: dx, dz and the weight's gradient over 262144 rows
        {"name": "norm_gate_train_bwd", "op": "norm", "dir": "bwd", "tokens": 8192, "heads": 32, "dim": 128,
         "act": "silu", "residual": False},
        # rotary positions of one decode step, a quarter of each head rotated, far into the context
        {"name": "rope_decode", "op": "rope", "dir": "fwd", "tokens": 256, "hq": 32, "hkv": 4, "dim": 128,
         "rotary": 32, "interleaved": False, "max_pos": 131072, "packed": True},
        # the gradient of the rotation over a long training sequence, neighbouring pairs, the whole head
        {"name": "rope_train_bwd", "op": "rope", "dir": "bwd", "tokens": 65536, "hq": 32, "hkv": 4, "dim": 128,
         "rotary": 128, "interleaved": True, "max_pos": 65536, "packed": False},
        # one decode step of 256 requests: a new page for the few that cross a page's end
        {"name": "plan_decode", "op": "plan", "requests": 256, "cached_lo": 1, "cached_hi": 8192, "new_lo": 1,
         "new_hi": 1, "page": 64},
        # a step that prefills 1024 requests of mixed lengths at once, small pages
        {"name": "plan_prefill", "op": "plan", "requests": 1024, "cached_lo": 0, "cached_hi": 4096, "new_lo": 0,
         "new_hi": 512, "page": 16},
        # the cache's write in a decode step: one token for each request, into pages that are partly full
        {"name": "append_decode", "op": "append", "requests": 256, "cached_lo": 1, "cached_hi": 1024, "new_lo": 1,
         "new_hi": 1, "hkv": 4, "dim": 128, "page": 64, "packed": True},
        # the cache's write of a long prefill, 65536 tokens of 8 requests whose last pages are partly full
        {"name": "append_prefill", "op": "append", "requests": 8, "cached_lo": 1, "cached_hi": 300, "new_lo": 8192,
         "new_hi": 8192, "hkv": 4, "dim": 128, "page": 64, "packed": False},
        # one request alone, one token: latency
        {"name": "attn_decode_one", "op": "attn", "requests": 1, "ctx_lo": 4096, "ctx_hi": 4096, "new_lo": 1,
         "new_hi": 1, "hq": 32, "hkv": 4, "dim": 128, "page": 64},
        # a serving batch of ragged contexts, one token each
        {"name": "attn_decode_ragged", "op": "attn", "requests": 256, "ctx_lo": 64, "ctx_hi": 8192, "new_lo": 1,
         "new_hi": 1, "hq": 32, "hkv": 4, "dim": 128, "page": 64},
        # few requests with very long contexts, four drafted tokens each (multi-token decode)
        {"name": "attn_draft_long", "op": "attn", "requests": 4, "ctx_lo": 130000, "ctx_hi": 131072, "new_lo": 4,
         "new_hi": 4, "hq": 32, "hkv": 4, "dim": 128, "page": 64},
        # a chunk of a long prompt: 4096 new tokens over 16384 in the cache, causal
        {"name": "attn_prefill", "op": "attn", "requests": 1, "ctx_lo": 16384, "ctx_hi": 16384, "new_lo": 4096,
         "new_hi": 4096, "hq": 32, "hkv": 4, "dim": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    """A whole number, spread over its logarithm, odd ones among them."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "plan", "append", "attn", "attn"])
    if op == "norm":
        if rng.random() < 0.5:  # the norm after a block, one head a row
            heads, dim = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 96, 128, 256])
        else:  # the norm before a block, one token a row
            heads, dim = 1, rng.choice([1000, 2048, 4096, 5120, 8192])
        tokens = _log(rng, 1, max(1, (8192 * 32 * 128) // (heads * dim * 2)))
        return {"op": "norm", "dir": rng.choice(["fwd", "bwd"]), "tokens": tokens, "heads": heads, "dim": dim,
                "act": rng.choice(["none", "silu", "sigmoid"]), "residual": rng.random() < 0.5}
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128, 256])
        hq = hkv * rng.choice([1, 2, 4, 8])
        return {"op": "rope", "dir": rng.choice(["fwd", "bwd"]), "tokens": _log(rng, 1, 65536 * 36 * 128 // ((hq + hkv) * dim)),
                "hq": hq, "hkv": hkv, "dim": dim, "rotary": rng.choice([dim, dim // 2, dim // 4]),
                "interleaved": rng.random() < 0.5, "max_pos": _log(rng, 128, 262144), "packed": rng.random() < 0.5}
    if op == "plan":
        requests = _log(rng, 1, 1024)
        return {"op": "plan", "requests": requests, "cached_lo": 0, "cached_hi": _log(rng, 1, 4096), "new_lo": rng.choice([0, 1]),
                "new_hi": _log(rng, 1, 512), "page": rng.choice([16, 32, 64, 128])}
    hkv, dim, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        requests = _log(rng, 1, 256)
        return {"op": "append", "requests": requests, "cached_lo": rng.choice([0, 1]), "cached_hi": _log(rng, 1, 1024),
                "new_lo": 1, "new_hi": _log(rng, 1, max(1, 2 * 65536 * 4 * 128 // (requests * hkv * dim * 2))), "hkv": hkv, "dim": dim,
                "page": page, "packed": rng.random() < 0.5}
    group = rng.choice([1, 2, 4, 7, 8])
    if rng.random() < 0.6:  # decode, one or a few tokens
        new = rng.choice([1, 1, 2, 4])
        requests = _log(rng, 1, 256)
        ctx = _log(rng, new, max(new, min(131072, 256 * 8192 * 4 * 128 // (requests * hkv * dim))))
        return {"op": "attn", "requests": requests, "ctx_lo": max(new, ctx // 8), "ctx_hi": ctx, "new_lo": new, "new_hi": new,
                "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page}
    requests = _log(rng, 1, 16)  # prefill, lengths mixed
    most = (32 * 4096 * 16384) // 2 // (requests * hkv * group)  # of new x context for one request
    new = _log(rng, 2, max(2, min(4096, int(math.sqrt(most)))))
    ctx = _log(rng, new, max(new, min(32768, most // new)))
    return {"op": "attn", "requests": requests, "ctx_lo": new, "ctx_hi": ctx, "new_lo": max(1, new // 4), "new_hi": new,
            "hq": hkv * group, "hkv": hkv, "dim": dim, "page": page}


def _spread(lo, hi, count):
    """`count` whole numbers over [lo, hi], the same for every seed; the first is hi."""
    return [hi - int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0) * 0.999999) for i in range(count)]


def _lengths(case):
    """(tokens in the cache before the step, new tokens) of each request."""
    n = case["requests"]
    new = _spread(case["new_lo"], case["new_hi"], n)
    if case["op"] == "attn":  # the context holds the new tokens already
        return [max(0, c - m) for c, m in zip(_spread(case["ctx_lo"], case["ctx_hi"], n), new)], new
    return _spread(case["cached_lo"], case["cached_hi"], n), new


# --------------------------------------------------------------- quantising
def _exponents(amax):
    """The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8 is the largest value of the 8-bit format), at least EXP_MIN."""
    mant, exp = torch.frexp(amax)  # amax = mant * 2^exp, mant in [0.5, 1)
    e = exp - 9 + (mant > 0.875).to(exp.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(min=EXP_MIN)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


# ----------------------------------------------------------------- prepare
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    r = random.Random(int(seed))
    bf = torch.bfloat16

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(case)
    op = case["op"]
    if op == "norm":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        shape = (T, H, D) if H > 1 else (T, D)
        s["x"] = (2.0 * randn(*shape)).to(bf)
        s["weight"] = 1.0 + 0.1 * randn(D)
        s["z"] = randn(*shape).to(bf) if case["act"] != "none" else None
        s["res"] = (2.0 * randn(*shape)).to(bf) if case["residual"] else None
        s["res_scale"] = 0.5 if case["residual"] else 1.0
        s["eps"] = 1e-6
        if case["dir"] == "bwd":
            s["dy"] = randn(*shape).to(bf)
            s["dh"] = randn(*shape).to(bf) if case["residual"] else None
        return s
    if op == "rope":
        T, hq, hkv, D, rot = case["tokens"], case["hq"], case["hkv"], case["dim"], case["rotary"]
        if case["packed"]:  # q and k as they leave a packed projection: views with a longer token stride
            qkv = randn(T, (hq + 2 * hkv) * D).to(bf)
            s["q"] = qkv[:, :hq * D].view(T, hq, D)
            s["k"] = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
        else:
            s["q"], s["k"] = randn(T, hq, D).to(bf), randn(T, hkv, D).to(bf)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(dev)
        if case["dir"] == "bwd":
            s["positions"] = (torch.arange(T, device=dev, dtype=torch.int32) + r.randrange(64)) % case["max_pos"]
        else:
            s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device=dev, dtype=torch.int32)
        s["factor"] = 1.0 if case["rotary"] == D else 1.2079441541679836  # scaled rotations lengthen q and k a little
        return s

    # operators of the paged cache
    bs = case["page"]
    cached, new = _lengths(case)
    pairs = list(zip(cached, new))
    r.shuffle(pairs)
    cached, new = [c for c, _ in pairs], [m for _, m in pairs]
    N, T = len(new), sum(new)
    total = [c + m for c, m in zip(cached, new)]
    have = [-(-c // bs) for c in (cached if op == "plan" else total)]
    need = [-(-t // bs) for t in total]
    width = max(1, max(need))
    pages = sum(need) + max(4, sum(need) // 16)
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int32)
    base = [0]
    for h in have:
        base.append(base[-1] + h)
    col = torch.arange(width, device=dev, dtype=torch.int32)[None, :]
    at = ints(base[:-1])[:, None] + col
    s["block_table"] = torch.where(col < ints(have)[:, None], order[at.clamp(max=pages - 1).long()], torch.full_like(at, -1))
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s["cu_seqlens"], s["cached_lens"], s["seq_lens"] = ints(cu), ints(cached), ints(total)
    s["tokens"], s["max_new"], s["max_ctx"] = T, max(new), max(total)
    if op == "plan":
        s["free_pages"] = order[base[-1]:].contiguous()
        s["num_free"] = ints([pages - base[-1]])
        return s
    hkv, D = case["hkv"], case["dim"]

    def cache():
        x = randn(pages, hkv, bs, D) * torch.exp(0.5 * randn(pages, hkv, 1, 1))
        x = x * torch.exp(0.25 * randn(1, hkv, 1, D))
        e = _exponents(x.abs().amax(dim=(2, 3)))
        return (x * _pow2(-e)[:, :, None, None]).to(F8), _pow2(e)

    s["k_cache"], s["k_scale"] = cache()
    s["v_cache"], s["v_scale"] = cache()
    if op == "append":
        if case["packed"]:
            kv = randn(T, 2 * hkv * D).to(bf)
            s["k"], s["v"] = kv[:, :hkv * D].view(T, hkv, D), kv[:, hkv * D:].view(T, hkv, D)
        else:
            s["k"], s["v"] = randn(T, hkv, D).to(bf), randn(T, hkv, D).to(bf)
        s["k"].mul_(2.0)
        tok = torch.arange(T, device=dev)
        req = torch.repeat_interleave(torch.arange(N, device=dev), ints(new).long(), output_size=T)
        pos = s["cached_lens"].long()[req] + tok - s["cu_seqlens"].long()[req]
        s["slots"] = (s["block_table"][req, pos // bs].long() * bs + pos % bs).int()
        return s
    s["q"] = randn(T, case["hq"], D).to(bf)
    s["scale"] = D ** -0.5
    return s


# --------------------------------------------------------------------- run
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_norm(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    act = None if s["act"] == "none" else s["act"]
    if s["dir"] == "fwd":
        return gdn.gdn_norm_gate(s["x"], s["weight"], residual=s["res"], z=s["z"], activation=act, eps=s["eps"],
                                 res_scale=s["res_scale"])
    return gdn.gdn_norm_gate_bwd(s["dy"], s["x"], s["weight"], z=s["z"], dh=s["dh"], activation=act, eps=s["eps"],
                                 res_scale=s["res_scale"])


def _own_rope(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn.gdn_rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=s["interleaved"],
                        attention_factor=s["factor"], inverse=s["dir"] == "bwd")


def _own_plan(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    got = gdn.gdn_paged_plan(s["cached_lens"], s["cu_seqlens"], s["block_table"], s["free_pages"], s["num_free"],
                             s["page"], s["tokens"])
    return (s["block_table"],) + tuple(got)  # seq_lens, slot_mapping, positions, the pages left


def _own_append(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    gdn.gdn_kv8_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _own_attn(s):
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn.gdn_kv8_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                 s["seq_lens"], cu_seqlens=s["cu_seqlens"], max_q_len=s["max_new"],
                                 max_seq_len=s["max_ctx"], scale=s["scale"])


def _act(z, act):
    sig = 1.0 / (1.0 + torch.exp(-z))
    return sig if act == "sigmoid" else z * sig


def _plain_norm(s):
    x, w = s["x"].float(), s["weight"]
    if s["dir"] == "fwd":
        h = x if s["res"] is None else s["res"].float() + s["res_scale"] * x
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * w
        if s["z"] is not None:
            y = y * _act(s["z"].float(), s["act"])
        return y.to(torch.bfloat16), None if s["res"] is None else h.to(torch.bfloat16)
    # x is the normed stream here
    dy = s["dy"].float()
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    n = x * rstd
    gate, dz = 1.0, None
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        gate = sig if s["act"] == "sigmoid" else z * sig
        slope = sig * (1.0 - sig) if s["act"] == "sigmoid" else sig * (1.0 + z * (1.0 - sig))
        dz = (dy * n * w * slope).to(torch.bfloat16)
    dyg = dy * gate
    dn = dyg * w
    dh = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
    dw = (dyg * n).reshape(-1, n.shape[-1]).sum(0)
    dres = dh.to(torch.bfloat16) if s["dh"] is not None else None
    return (s["res_scale"] * dh).to(torch.bfloat16), dres, dz, dw


def _rotate(x, cos, sin, rot, interleaved):
    part = x[..., :rot].float()
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned.to(x.dtype), x[..., rot:]), -1)


def _plain_rope(s):
    angle = s["positions"].float()[:, None, None] * s["inv_freq"]
    cos, sin = torch.cos(angle) * s["factor"], torch.sin(angle) * s["factor"]
    if s["dir"] == "bwd":
        sin = -sin
    return (_rotate(s["q"], cos, sin, s["rotary"], s["interleaved"]), _rotate(s["k"], cos, sin, s["rotary"], s["interleaved"]))


def _plain_plan(s):
    bs, cu, cached, table = s["page"], s["cu_seqlens"].long(), s["cached_lens"].long(), s["block_table"]
    lens = cached + cu[1:] - cu[:-1]
    have, need = (cached + bs - 1) // bs, (lens + bs - 1) // bs
    want = need - have
    first = torch.cumsum(want, 0) - want  # pages that the requests before take
    left = s["num_free"].long()
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    index = left - 1 - (first[:, None] + col - have[:, None])  # taken from the end of the free list
    fresh = (col >= have[:, None]) & (col < need[:, None])
    page = s["free_pages"][index.clamp(0, s["free_pages"].shape[0] - 1)].long()
    page = torch.where(index >= 0, page, torch.full_like(index, -1))
    table.copy_(torch.where(fresh, page, table.long()))
    tok = torch.arange(s["tokens"], device=table.device)
    req = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = cached[req] + tok - cu[req]
    at = table[req, pos // bs].long()
    slots = torch.where(at >= 0, at * bs + pos % bs, torch.full_like(at, -1))
    return table, lens.int(), slots.int(), pos.int(), (left - torch.minimum(want.sum(), left)).int()


def _append_one(x, cache, scale, slots):
    bs, D = cache.shape[2], cache.shape[3]
    page, off = slots.long() // bs, slots.long() % bs
    P, H = scale.shape
    index = page[:, None].expand(-1, H)
    x = x.float()
    amax = torch.zeros(P, H, device=x.device).scatter_reduce(0, index, x.abs().amax(-1), "amax")
    start = torch.full((P,), bs, device=x.device).scatter_reduce(0, page, off, "amin")  # first new place in each page
    old = (torch.frexp(scale)[1] - 1)
    kept = torch.where((start == 0)[:, None], torch.full_like(old, EXP_MIN), old)
    e = torch.where((start < bs)[:, None], torch.maximum(kept, _exponents(amax)), old)
    before = torch.arange(bs, device=x.device)[None, :] < torch.where(start < bs, start, torch.zeros_like(start))[:, None]
    shift = torch.where(before[:, None, :], (old - e)[:, :, None], torch.zeros_like(old)[:, :, None])
    codes = (cache.float() * _pow2(shift)[..., None]).to(F8)
    put = (x * _pow2(-e[page])[..., None]).to(F8)
    codes = codes.view(torch.uint8)
    codes[page[:, None], torch.arange(H, device=x.device)[None, :], off[:, None]] = put.view(torch.uint8)
    cache.view(torch.uint8).copy_(codes)
    scale.copy_(_pow2(e))


def _plain_append(s):
    _append_one(s["k"], s["k_cache"], s["k_scale"], s["slots"])
    _append_one(s["v"], s["v_cache"], s["v_scale"], s["slots"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_attn(s):
    table, bs, D = s["block_table"].long().clamp(min=0), s["page"], s["dim"]
    N, hkv, G, M = table.shape[0], s["hkv"], s["hq"] // s["hkv"], s["max_new"]
    cu, lens = s["cu_seqlens"].long(), s["seq_lens"].long()

    def values(cache, scale):  # [N, hkv, places, D]
        got = cache.view(torch.uint8)[table].view(F8).float() * scale[table][..., None, None]
        return got.permute(0, 2, 1, 3, 4).reshape(N, hkv, -1, D)

    k = values(s["k_cache"], s["k_scale"])
    i = torch.arange(M, device=k.device)
    count = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=s["tokens"] - 1)  # [N, M], rows past a request's own are not kept
    q = s["q"].float()[at].view(N, M, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(N, hkv, M * G, D)
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    del k
    limit = lens[:, None] - count[:, None] + i  # the last place that row i sees
    seen = (torch.arange(p.shape[-1], device=p.device) <= limit[..., None]).repeat_interleave(G, 1)[:, None]
    p.masked_fill_(~seen, -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    v = values(s["v_cache"], s["v_scale"])
    o = torch.matmul(p, v) / total
    o = o.view(N, hkv, M, G, D).permute(0, 2, 1, 3, 4).reshape(N, M, hkv * G, D)
    keep = (i < count[:, None]).reshape(-1).nonzero()[:, 0] if s["new_lo"] != s["new_hi"] else slice(None)
    return o.reshape(N * M, hkv * G, D)[keep].to(torch.bfloat16)


_own = {"norm": _own_norm, "rope": _own_rope, "plan": _own_plan, "append": _own_append, "attn": _own_attn}
_plain = {"norm": _plain_norm, "rope": _plain_rope, "plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "norm":
        D = case["dim"]
        n = case["tokens"] * case["heads"] * D
        tensors = 2 + (case["act"] != "none") + 2 * case["residual"]  # x, y; z; residual, h
        if case["dir"] == "bwd":  # dy, x, dx; z, dz; dh, dres
            tensors = 3 + 2 * (case["act"] != "none") + 2 * case["residual"]
        return {"bytes": 2 * tensors * n + 4 * D * (1 if case["dir"] == "fwd" else 2), "flops": 8 * n}
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"] + 2 * case["rotary"], "flops": 3 * n}
    cached, new = _lengths(case)
    T, bs = sum(new), case["page"]
    if op == "plan":
        grown = sum(-(-(c + m) // bs) - -(-c // bs) for c, m in zip(cached, new))
        # lengths and offsets in, lengths out; a table entry and a free page for each page taken; of the tables, the
        # page that each request's first new token goes to; slot and position of each token
        return {"bytes": 4 * (3 * len(new) + 1) + 8 * grown + 4 * len(new) + 8 * T + 8, "flops": 8 * T}
    hkv, D = case["hkv"], case["dim"]
    if op == "append":
        pages = sum(-(-(c + m) // bs) - c // bs for c, m in zip(cached, new) if m)
        return {"bytes": T * hkv * D * 2 * 3 + 4 * T + pages * hkv * 16, "flops": 4 * T * hkv * D}
    G = case["hq"] // hkv
    places = sum(c + m for c, m in zip(cached, new))
    pairs = sum(m * c + m * (m + 1) // 2 for c, m in zip(cached, new))
    pages = sum(-(-(c + m) // bs) for c, m in zip(cached, new))
    return {"bytes": 2 * places * hkv * D + pages * (8 * hkv + 4) + 4 * T * case["hq"] * D, "flops": 4 * pairs * hkv * G * D}


# ------------------------------------------------------------------- exact
def _to8(x):
    """x rounded to the 8-bit format's values: three bits after the leading one, steps of 2^-9 below 2^-6, ties to even."""
    exp = torch.frexp(x)[1].clamp(min=-5)
    step = torch.ldexp(torch.ones_like(x), exp - 4)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits; None for the plan, whose outputs are whole numbers."""
    if case["op"] == "plan":
        return None

    def norm(s):
        f = torch.float64
        w = s["weight"].to(f)
        x = s["x"].to(f)
        sig = torch.sigmoid(s["z"].to(f)) if s["z"] is not None else None
        gate = 1.0 if sig is None else sig if s["act"] == "sigmoid" else sig * s["z"].to(f)
        if s["dir"] == "fwd":
            h = x if s["res"] is None else torch.add(s["res"].to(f), x, alpha=s["res_scale"])
            rms = h.square().mean(-1, keepdim=True).add(s["eps"]).sqrt()
            return (h / rms) * (w * gate), None if s["res"] is None else h
        D = x.shape[-1]
        inv = x.square().mean(-1, keepdim=True).add(s["eps"]).rsqrt()
        up = s["dy"].to(f) * gate * w
        dot = (up * x).sum(-1, keepdim=True)
        dh = up * inv - x * (dot * inv ** 3 / D)
        if s["dh"] is not None:
            dh = dh + s["dh"].to(f)
        dz = None
        if sig is not None:
            d = sig * (1 - sig)
            if s["act"] != "sigmoid":
                d = sig + s["z"].to(f) * d
            dz = s["dy"].to(f) * w * (x * inv) * d
        dw = torch.einsum("rd,rd->d", (s["dy"].to(f) * gate).reshape(-1, D), (x * inv).reshape(-1, D))
        return s["res_scale"] * dh, dh if s["dh"] is not None else None, dz, dw

    def rope(s):
        f, rot = torch.float64, s["rotary"]
        sign = -1.0 if s["dir"] == "bwd" else 1.0
        angle = torch.outer(s["positions"].to(f), s["inv_freq"].to(f)) * sign
        turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]

        def one(x):
            x = x.to(f)
            a = x[..., 0:rot:2] if s["interleaved"] else x[..., :rot // 2]
            b = x[..., 1:rot:2] if s["interleaved"] else x[..., rot // 2:rot]
            c = torch.complex(a.contiguous(), b.contiguous()) * turn
            y = x.clone()
            if s["interleaved"]:
                y[..., 0:rot:2], y[..., 1:rot:2] = c.real, c.imag
            else:
                y[..., :rot // 2], y[..., rot // 2:rot] = c.real, c.imag
            return y

        return one(s["q"]), one(s["k"])

    def append(s):
        def one(x, cache, scale):
            bs = cache.shape[2]
            x = x.double().cpu()
            codes, exps = cache.double().cpu(), torch.log2(scale.double()).round().int().cpu()
            runs = []  # (page, first place, first token, count)
            for t, slot in enumerate(s["slots"].tolist()):
                if runs and runs[-1][0] == slot // bs and runs[-1][1] + runs[-1][3] == slot % bs:
                    runs[-1][3] += 1
                else:
                    runs.append([slot // bs, slot % bs, t, 1])
            for page, off, t, n in runs:
                new = x[t:t + n].transpose(0, 1)  # [heads, n, D]
                amax = new.abs().amax((1, 2))
                e = torch.where(amax > 0, torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0)), torch.tensor(float(EXP_MIN), dtype=torch.float64))
                e = torch.maximum(e, torch.tensor(float(EXP_MIN), dtype=torch.float64))
                if off:
                    e = torch.maximum(e, exps[page].double())
                    codes[page, :, :off] = _to8(codes[page, :, :off] * torch.exp2(exps[page].double() - e)[:, None, None])
                codes[page, :, off:off + n] = _to8(new * torch.exp2(-e)[:, None, None])
                exps[page] = e.int()
            return codes, torch.exp2(exps.double())

        k, ks = one(s["k"], s["k_cache"], s["k_scale"])
        v, vs = one(s["v"], s["v_cache"], s["v_scale"])
        return k, v, ks, vs

    def attn(s):
        f, bs, D, hkv = torch.float64, s["page"], s["dim"], s["hkv"]
        G = s["hq"] // hkv
        lens, cu = s["seq_lens"].tolist(), s["cu_seqlens"].tolist()
        out = torch.zeros(s["tokens"], s["hq"], D, dtype=f, device=s["q"].device)
        for n, L in enumerate(lens):
            m = cu[n + 1] - cu[n]
            pages = s["block_table"][n, :-(-L // bs)].long()
            for h in range(hkv):
                k = (s["k_cache"].view(torch.uint8)[pages, h].view(F8).to(f) * s["k_scale"][pages, h].to(f)[:, None, None]).reshape(-1, D)[:L]
                v = (s["v_cache"].view(torch.uint8)[pages, h].view(F8).to(f) * s["v_scale"][pages, h].to(f)[:, None, None]).reshape(-1, D)[:L]
                for i in range(0, m, 512):  # rows at once
                    rows = slice(cu[n] + i, cu[n] + min(i + 512, m))
                    q = s["q"][rows, h * G:(h + 1) * G].to(f)
                    a = torch.einsum("tgd,kd->tgk", q, k) * s["scale"]
                    last = L - m + i + torch.arange(q.shape[0], device=a.device)
                    a = a.masked_fill((torch.arange(L, device=a.device) > last[:, None])[:, None, :], -math.inf)
                    out[rows, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", torch.softmax(a, -1), v)
        return out

    return {"norm": norm, "rope": rope, "append": append, "attn": attn}[case["op"]](prepare(case, seed))
