"""A training step's attention on the GPU against plain 64-bit implementations (tests/train_util.py).

Tolerances, from the roundings.  A bf16 result is off by half a step, 2^-8 of its value.  The softmax weights, and the
gradients of the logits, enter the products in bf16: 2^-8 of each term, so 2^-8 of the sum of the terms' magnitudes.
What stays in fp32: a logit is a sum of D products, off by some D 2^-24 = 2^-17 of the sum of their magnitudes M (the
tensor cores may cut instead of round, twice that), and that is the relative error of its weight, beside 2^-21 of the
hardware's exponential; delta and dP likewise.  2^-15 (1 + M) of the terms' magnitudes covers their sum.  The gradient
takes o in bf16, as the forward gave it: delta is off by 2^-8 sum |do o|, which is a term like the rounded ones."""
import math

import numpy as np
import pytest
import torch

import stack_util as S
import train_util as U

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_chunked_chunk_gb300 import build
    build.build()


def _gdn():
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn


def _inputs(lens, lens_k, HQ, HK, D, seed, packed=True, q_size=2.0):
    g = torch.Generator().manual_seed(seed)
    Tq, Tk = sum(lens), sum(lens if lens_k is None else lens_k)
    q, k, v, do = (torch.randn(t, h, D, generator=g) for t, h in ((Tq, HQ), (Tk, HK), (Tk, HK), (Tq, HQ)))
    return (q_size * q).to(BF), k.to(BF), v.to(BF), do.to(BF)


def _gpu(q, k, v, packed):
    """On the GPU; packed: views of one projection's output."""
    if not packed or q.shape[0] != k.shape[0]:
        return q.cuda(), k.cuda(), v.cuda()
    T, D = q.shape[0], q.shape[2]
    w = torch.cat([t.reshape(T, -1) for t in (q, k, v)] + [torch.full((T, 8), math.nan, dtype=BF)], 1).cuda()
    return tuple(t.unflatten(1, (-1, D)) for t in w[:, :-8].split([q.shape[1] * D, k.shape[1] * D, v.shape[1] * D], 1))


def _near(got, ref, tol, what):
    got = got.double().cpu()
    assert not torch.isnan(got).any(), what
    over = (got - ref).abs() - tol
    over[got == ref] = -1.0  # infinities
    assert (over <= 0).all(), f"{what}: {(over > 0).sum()} of {over.numel()}, worst {over.max():.3e} at {over.argmax()}"


def _check_fwd(o, lse, r):
    _near(o, r["o"], 2.0 ** -8 * r["o"].abs() + (2.0 ** -8 + 2.0 ** -15 * r["lse_mag"][..., None]) * r["o_mag"] + 1e-30, "o")
    _near(lse, r["lse"], 2.0 ** -15 * r["lse_mag"] + 2.0 ** -22 * r["lse"].abs().nan_to_num(0, 0, 0), "lse")


def _check_bwd(grads, r):
    for x, n in zip(grads, ("dq", "dk", "dv")):
        tol = 2.0 ** -8 * r[n].abs() + 2.0 ** -8 * r[n + "_round"] + 2.0 ** -15 * r[n + "_fp32"] + 1e-30
        if n != "dv":  # delta from the rounded o
            tol = tol + 2.0 ** -8 * r[n + "_delta"]
        _near(x, r[n], tol, n)


def _run(lens, lens_k, HQ, HK, D, causal, seed, packed=True, scale=None, bwd=True, q_size=2.0):
    gdn = _gdn()
    q, k, v, do = _inputs(lens, lens_k, HQ, HK, D, seed, q_size=q_size)
    cq, ck, cv = _gpu(q, k, v, packed)
    cu = U.offsets(lens).cuda()
    cu_k = None if lens_k is None else U.offsets(lens_k).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(cu_seqlens=cu, cu_seqlens_k=cu_k, causal=causal, scale=scale, dev_status=status)
    o, lse = gdn.gdn_attention_fwd(cq, ck, cv, **args)
    r = U.attention(q, k, v, U.spans(lens, lens_k), causal, D ** -0.5 if scale is None else scale, do)
    assert int(status) == 0
    _check_fwd(o, lse, r)
    if bwd:
        grads = gdn.gdn_attention_bwd(do.cuda(), cq, ck, cv, o, lse, **args)
        assert int(status) == 0
        _check_bwd(grads, r)
    return o, lse


SIZES = [  # lens, lens_k, HQ, HK, D
    ([128], None, 1, 1, 128), ([1], None, 2, 1, 64), ([127], None, 1, 1, 64), ([129], None, 3, 1, 128), ([256], None, 8, 2, 128),
    ([257, 1, 0, 383], None, 2, 2, 64), ([5, 130, 64, 1, 300], None, 7, 1, 128), ([512], None, 2, 1, 128),
    ([640, 100], None, 2, 2, 128), ([1000], None, 1, 1, 64),
    ([100, 200], [300, 200], 2, 1, 128), ([1, 1, 1], [1, 700, 128], 4, 2, 64), ([300, 40], [100, 0], 2, 2, 128),
    ([0, 129], [50, 257], 1, 1, 128), ([200], [129], 2, 2, 64),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_forward(case, causal):
    _run(*SIZES[case], causal, case, bwd=False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_gradients(case, causal):
    _run(*SIZES[case], causal, 100 + case)


# ----------------------------------------------------- activations in 8 bits
# Codes, scales and their values are exact: they are compared for equality.

def _codes(x):
    """Values of the codes, and scales, of a float64 array [rows, D] by the definition."""
    rows, D = x.shape
    codes, scale = np.zeros_like(x), np.zeros((rows, -(-D // 128)))
    for r in range(rows):
        for g in range(scale.shape[1]):
            part = x[r, 128 * g:128 * g + 128]
            fin = np.abs(part[np.isfinite(part)])
            e = S.least_exponent(float(fin.max()) if fin.size else 0.0)
            scale[r, g] = 2.0 ** e
            codes[r, 128 * g:128 * g + 128] = np.where(np.isfinite(part), S.to_e4m3(np.where(np.isfinite(part), part, 0) * 2.0 ** -e), np.nan)
    return codes, scale


def _same(got, ref):
    np.testing.assert_array_equal(S.f64(got).reshape(ref.shape), ref)


@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 64), (7, 96), (33, 128), (4, 3, 136), (2, 5, 1000), (3, 4096), (9, 130), (1000, 8),
                                   (2, 257), (70, 1, 256)])
def test_act8(shape):
    gdn = _gdn()
    g = torch.Generator().manual_seed(sum(shape))
    x = (torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape[:-1] + (1,), generator=g))).to(BF)
    codes, scale = gdn.gdn_act8_save(x.cuda())
    ref, rs = _codes(S.f64(x).reshape(-1, shape[-1]))
    assert codes.shape == x.shape and scale.shape == x.shape[:-1] + (-(-shape[-1] // 128),)
    _same(codes, ref)
    _same(scale, rs)
    y = gdn.gdn_act8_load(codes, scale)
    _same(y, ref * np.repeat(rs, 128, 1)[:, :shape[-1]])
    # from a slice of a wider tensor, and into buffers of the caller's
    wide = torch.full(shape[:-1] + (shape[-1] + 24,), math.nan, dtype=BF)
    wide[..., 8:8 + shape[-1]] = x
    part = wide.cuda()[..., 8:8 + shape[-1]]
    if len(shape) == 2:
        c2, s2 = torch.empty_like(codes), torch.empty_like(scale)
        assert gdn.gdn_act8_save(part, codes=c2, scale=s2)[0] is not None
        assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)


def test_act8_of_heads_within_a_token_and_of_odd_addresses():
    gdn = _gdn()
    g = torch.Generator().manual_seed(5)
    w = torch.randn(37, 4 * 96 + 16, generator=g).to(BF).cuda()
    x = w[:, 16:].unflatten(1, (4, 96))
    codes, scale = gdn.gdn_act8_save(x)
    ref, rs = _codes(S.f64(x).reshape(-1, 96))
    _same(codes, ref)
    _same(scale, rs)
    odd = torch.empty(x.numel() + 1, dtype=BF, device="cuda")[1:].view(37, 4, 96)  # 2-byte aligned
    odd.copy_(x)
    c2, s2 = gdn.gdn_act8_save(odd)
    assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scale)
    c3 = torch.empty(codes.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(codes.shape)
    c3.copy_(codes.view(torch.uint8))
    assert torch.equal(gdn.gdn_act8_load(c3.view(torch.float8_e4m3fn), scale, out=torch.empty_like(odd)), gdn.gdn_act8_load(codes, scale))


@pytest.mark.parametrize("D", [128, 100, 8])
def test_act8_of_extremes(D):
    gdn = _gdn()
    x = torch.zeros(9, D)
    x[1, 0], x[1, 1] = math.inf, 1.0
    x[2, 3], x[2, 4] = -math.inf, math.nan
    x[3] = math.nan
    x[4, 0], x[4, 5] = 3.3895313892515355e38, -1.0  # the largest bf16
    x[5, 0], x[5, 1] = 1e-38, 9.2e-41               # below what the smallest scale holds
    x[6, 0], x[6, 1] = 448.0, 449.0
    x[7, 0] = -448.0
    x[8] = torch.linspace(-1.0, 1.0, D)
    x = x.to(BF)
    codes, scale = gdn.gdn_act8_save(x.cuda())
    ref, rs = _codes(S.f64(x))
    _same(codes, ref)
    _same(scale, rs)
    _same(gdn.gdn_act8_load(codes, scale), S.f64(torch.from_numpy(ref * rs).to(BF)))


NORM_SHAPES = [(1, 128), (257, 2, 128), (33, 4, 64), (5, 3, 96), (130, 256), (9, 512), (5, 1000), (7, 1024), (5, 2048), (3, 4096), (3, 8192),
               (2, 16384), (1000, 8)]


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("kind,res", [(None, False), ("silu", True), ("sigmoid", False), (None, True)])
def test_norm_gate_with_codes(shape, kind, res):
    gdn = _gdn()
    g = torch.Generator().manual_seed(sum(shape))
    x = (2 * torch.randn(shape, generator=g)).to(BF)
    w = 1 + 0.1 * torch.randn(shape[-1], generator=g)
    z = torch.randn(shape, generator=g).to(BF) if kind else None
    r = torch.randn(shape, generator=g).to(BF) if res else None
    dy, dh = torch.randn(shape, generator=g).to(BF), torch.randn(shape, generator=g).to(BF) if res else None
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    args = dict(activation=kind, res_scale=0.5 if res else 1.0)
    y, h, h8, hs, z8, zs = gdn.gdn_norm_gate_save8(c(x), c(w), residual=c(r), z=c(z), **args)
    ry, rh = S.norm_fwd(S.f64(x), S.f64(w), S.f64(r), S.f64(z), kind, res_scale=args["res_scale"])
    _near(y, torch.from_numpy(ry), 2.0 ** -8 * torch.from_numpy(np.abs(ry)) + 1e-37, "y")
    if res:
        _near(h, torch.from_numpy(rh), torch.from_numpy(2.0 ** -8 * np.abs(rh) + 2.0 ** -18 * np.abs(rh).max()), "h")
    assert (h is None) == (not res) and (z8 is None) == (zs is None) == (kind is None)
    for t, codes, scale in ((x if h is None else h, h8, hs), (z, z8, zs)):
        if t is not None:
            want = gdn.gdn_act8_save(t.cuda())
            assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scale, want[1])
    dx, dres, dz, dw = gdn.gdn_norm_gate_bwd8(c(dy), h8, hs, c(w), z_codes=z8, z_scale=zs, dh=c(dh), **args)
    h64 = S.f64(gdn.gdn_act8_load(h8, hs))  # exact: an e4m3 number and a power of two
    z64 = None if z is None else S.f64(gdn.gdn_act8_load(z8, zs))
    rx, rr, rz, rw = S.norm_bwd(S.f64(dy), h64, S.f64(w), z64, S.f64(dh), kind, res_scale=args["res_scale"])
    rstd = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + 1e-6)
    terms = rstd * np.abs(S.f64(dy)).max(-1, keepdims=True) * 4 + (2.0 if res else 0.0)
    n = h64 * rstd
    for got, ref, mag in ((dx, rx, terms), (dres, rr, terms), (dz, rz, np.abs(S.f64(dy) * n))):
        if got is not None:
            _near(got, torch.from_numpy(ref), torch.from_numpy(2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * mag + 1e-37), "gradient")
    assert (dres is None) == (not res) and (dz is None) == (kind is None)
    mags = np.abs(S.f64(dy) * n * (1.0 if kind is None else S.act(z64, kind)[0])).reshape(-1, shape[-1]).sum(0)
    assert (np.abs(S.f64(dw) - rw) <= 2.0 ** -19 * mags + 1e-30).all()
    again = gdn.gdn_norm_gate_bwd8(c(dy), h8, hs, c(w), z_codes=z8, z_scale=zs, dh=c(dh), **args)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dres, dz, dw)) if a is not None)


# ------------------------------------------------- attention, where it can go wrong
def _same_bits(a, b):
    return all(torch.equal(x.view(torch.int16) if x.dtype == BF else x.view(torch.int32), y.view(torch.int16) if y.dtype == BF else y.view(torch.int32))
               for x, y in zip(a, b))


def _all(q, k, v, do, **args):
    gdn = _gdn()
    o, lse = gdn.gdn_attention_fwd(q, k, v, **args)
    return (o, lse) + tuple(gdn.gdn_attention_bwd(do, q, k, v, o, lse, **args))


@pytest.mark.parametrize("D,HQ,HK", [(128, 4, 2), (64, 3, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences(D, HQ, HK, causal):
    """More sequences than a warp has lanes, empty ones among them, and keys of other lengths."""
    g = torch.Generator().manual_seed(D + HQ)
    lens = torch.randint(0, 160, (75,), generator=g).tolist()
    lens[10] = lens[70] = 0
    _run(lens, None, HQ, HK, D, causal, 7)
    lens_k = [max(0, m + d) for m, d in zip(lens, torch.randint(-40, 90, (75,), generator=g).tolist())]
    _run(lens, lens_k, HQ, HK, D, causal, 8)


@pytest.mark.parametrize("kind", ["grow", "fall", "equal", "large", "tiny"])
def test_running_maximum(kind):
    """Logits that grow along the keys by more than the reference may lag, fall, are all equal, large, or tiny."""
    T, D = 700, 128
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(T, 1, D, generator=g) for _ in range(4))
    u = torch.nn.functional.normalize(torch.randn(D, generator=g), dim=0)
    if kind in ("grow", "fall"):
        at = torch.arange(T)[:, None, None] / T * (60.0 if kind == "grow" else -60.0)
        q, k = q * 0.2 + u * D ** 0.5, k * 0.2 + at * u
    elif kind == "equal":
        k = k[:1].expand(T, 1, D).contiguous()
    else:
        q, k = (t * (30.0 if kind == "large" else 1e-3) for t in (q, k))
    q, k, v, do = (t.to(BF) for t in (q, k, v, do))
    r = U.attention(q, k, v, [(0, T, 0, T)], True, D ** -0.5, do)
    o, lse, *grads = _all(*(t.cuda() for t in (q, k, v, do)))
    _check_fwd(o, lse, r)
    _check_bwd(grads, r)


@pytest.mark.parametrize("scale", [0.5, 1e-4, 3.0])
def test_scale(scale):
    _run([130, 77], None, 2, 1, 64, True, 21, scale=scale)


@pytest.mark.parametrize("causal", [True, False])
def test_other_sequences_do_not_reach_one(causal):
    """NaN and infinities in the sequences before and after, whose rows share tiles with it, and in what stands between
    the heads' tokens: the same bits as without."""
    lens = [37, 201, 90]
    q, k, v, do = _inputs(lens, None, 4, 2, 128, 5)
    a, b = 37, 238
    clean = _all(*(t[a:b].contiguous().cuda() for t in (q, k, v, do)), causal=causal)
    for t in (q, k, v, do):
        t[:a:2], t[1:a:2], t[b:] = math.nan, math.inf, -math.inf
        t[b + 1::3] = math.nan
    cq, ck, cv = _gpu(q, k, v, True)
    dirty = _all(cq, ck, cv, do.cuda(), cu_seqlens=U.offsets(lens).cuda(), causal=causal)
    assert _same_bits([t[a:b] for t in dirty], clean)


def test_rows_behind_the_last_sequence_are_zero():
    lens, pad = [150, 20], 300
    q, k, v, do = _inputs(lens + [pad], None, 4, 2, 64, 6)
    for t in (q, k, v, do):
        t[170:] = math.nan
    cu = U.offsets(lens).cuda()
    got = _all(*(t.cuda() for t in (q, k, v, do)), cu_seqlens=cu)
    want = _all(*(t[:170].contiguous().cuda() for t in (q, k, v, do)), cu_seqlens=cu)
    assert _same_bits([t[:170] for t in got], want)
    assert (got[0][170:] == 0).all() and (got[1][170:] == -math.inf).all() and all((t[170:] == 0).all() for t in got[2:])


def test_no_rows_no_keys_no_sequences():
    gdn = _gdn()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new = lambda t, h: torch.randn(t, h, 64, device="cuda").to(BF)  # noqa: E731
    q, k, v = new(5, 2), new(7, 1), new(7, 1)
    # rows without keys
    o, lse, dq, dk, dv = _all(q, k[:0], v[:0], torch.ones_like(q), cu_seqlens=ints(0, 5), cu_seqlens_k=ints(0, 0))
    assert (o == 0).all() and (lse == -math.inf).all() and (dq == 0).all() and dk.shape == (0, 1, 64)
    # keys without rows
    o, lse, dq, dk, dv = _all(q[:0], k, v, q[:0], cu_seqlens=ints(0, 0), cu_seqlens_k=ints(0, 7))
    assert o.shape == (0, 2, 64) and dq.shape == (0, 2, 64) and (dk == 0).all() and (dv == 0).all()
    # no sequences at all
    o, lse, dq, dk, dv = _all(q, new(5, 1), new(5, 1), torch.ones_like(q), cu_seqlens=ints(0))
    assert (o == 0).all() and (lse == -math.inf).all() and all((t == 0).all() for t in (dq, dk, dv))
    # nothing
    assert gdn.gdn_attention_fwd(q[:0], k[:0], v[:0])[0].shape == (0, 2, 64)


def test_bad_offsets_are_reported():
    gdn = _gdn()
    q, k, v, do = (t.cuda() for t in _inputs([300], None, 2, 1, 64, 9))
    good = _all(q[:100], k[:100], v[:100], do[:100])
    for cu in ([0, 100, 90, 300], [0, 100, 400], [-1, 100, 300], [5, 100, 300], [0, 100, -7]):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = gdn.gdn_attention_fwd(q, k, v, cu_seqlens=c, dev_status=st)
        assert int(st) == gdn.DEV_BAD_CU_SEQLENS
        st.zero_()
        grads = gdn.gdn_attention_bwd(do, q, k, v, o, lse, cu_seqlens=c, dev_status=st)
        assert int(st) == gdn.DEV_BAD_CU_SEQLENS
        if cu == [0, 100, 400]:  # the good sequence gets its results
            assert _same_bits([o[:100], lse[:100]] + [t[:100] for t in grads], good)


def test_runs_agree_bit_for_bit():
    lens = [513, 260, 1000]
    q, k, v, do = (t.cuda() for t in _inputs(lens, None, 8, 2, 128, 11))
    cu = U.offsets(lens).cuda()
    a = _all(q, k, v, do, cu_seqlens=cu)
    for _ in range(3):
        assert _same_bits(a, _all(q, k, v, do, cu_seqlens=cu))


def test_two_streams_at_once():
    """Two calls at once on two streams, each with its own outputs and workspace."""
    gdn = _gdn()
    sets = [tuple(t.cuda() for t in _inputs([900, 300], None, 8, 2, 128, s)) for s in (1, 2)]
    cu = U.offsets([900, 300]).cuda()
    want = [_all(*s, cu_seqlens=cu) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for (q, k, v, do), st in zip(sets, streams):
        with torch.cuda.stream(st):
            o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
            ws = torch.empty(gdn.attention_bwd_workspace_size(2, 1200, 1200, 8, 2, 128), dtype=torch.uint8, device="cuda")
            for _ in range(4):
                gdn.gdn_attention_fwd(q, k, v, cu_seqlens=cu, o=o, lse=lse)
                grads = gdn.gdn_attention_bwd(do, q, k, v, o, lse, cu_seqlens=cu, workspace=ws)
            got.append((o, lse) + tuple(grads))
    torch.cuda.synchronize()
    assert all(_same_bits(a, b) for a, b in zip(want, got))


def test_captured_and_replayed_with_other_inputs():
    gdn = _gdn()
    a, b = (tuple(t.cuda() for t in _inputs([300, 45], None, 4, 1, 128, s)) for s in (1, 2))
    cu, cu_b = U.offsets([300, 45]).cuda(), U.offsets([20, 325]).cuda()
    want_a, want_b = _all(*a, cu_seqlens=cu), _all(*b, cu_seqlens=cu_b)
    held, held_cu = [t.clone() for t in a], cu.clone()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _all(*held, cu_seqlens=held_cu)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        out = _all(*held, cu_seqlens=held_cu)
        codes = gdn.gdn_act8_save(held[0])
        back = gdn.gdn_act8_load(*codes)
    graph.replay()
    assert _same_bits(out, want_a)
    for t, x in zip(held, b):
        t.copy_(x)
    held_cu.copy_(cu_b)
    graph.replay()
    assert _same_bits(out, want_b)
    assert torch.equal(back, gdn.gdn_act8_load(*gdn.gdn_act8_save(b[0])))


def test_offsets_past_32_bits():
    """Token strides and outputs whose offsets need more than 32 bits."""
    gdn = _gdn()
    T, D, ld = 700, 64, 4 << 20  # 2.9e9 elements from end to end
    base = torch.empty(T * ld, dtype=BF, device="cuda")
    q0, k0, v0, do = _inputs([T], None, 2, 1, D, 4)
    views = []
    for at, x in ((0, q0), (1024, k0), (2048, v0)):
        t = base.as_strided((T, x.shape[1], D), (ld, D, 1), at)
        t.copy_(x)
        views.append(t)
    got = _all(*views, do.cuda())
    assert _same_bits(got, _all(*(t.cuda() for t in (q0, k0, v0, do))))
    del base, views
    # many short sequences of many heads: 2.4e9 elements of q, o and their gradients
    lens, HQ = [37] * 640, 800
    T = sum(lens)
    q = torch.zeros(T, HQ, 128, dtype=BF, device="cuda")
    k, v = (torch.zeros(T, 2, 128, dtype=BF, device="cuda") for _ in range(2))
    do = torch.zeros_like(q)
    q1, k1, v1, do1 = _inputs([74], None, HQ, 2, 128, 14)
    for t, x in ((q, q1), (k, k1), (v, v1), (do, do1)):
        t[-74:].copy_(x)
    o, lse, dq, dk, dv = _all(q, k, v, do, cu_seqlens=U.offsets(lens).cuda())
    want = _all(*(t.cuda() for t in (q1, k1, v1, do1)), cu_seqlens=U.offsets([37, 37]).cuda())
    assert _same_bits([t[-74:] for t in (o, lse, dq)], want[:3])
    # (dk and dv are sums of parts, cut by the work of the whole batch: the same to rounding)
    r = U.attention(q1, k1, v1, U.spans([37, 37]), True, 128 ** -0.5, do1)
    _check_bwd([t[-74:] for t in (dq, dk, dv)], r)


def test_act8_past_32_bits():
    gdn = _gdn()
    x = torch.zeros(270000, 8192, dtype=BF, device="cuda")
    tail = torch.randn(3, 8192, generator=torch.Generator().manual_seed(1)).to(BF)
    x[-3:].copy_(tail)
    codes, scale = gdn.gdn_act8_save(x)
    want = gdn.gdn_act8_save(tail.cuda())
    assert torch.equal(codes[-3:].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scale[-3:], want[1])
    del x
    assert torch.equal(gdn.gdn_act8_load(codes, scale)[-3:], gdn.gdn_act8_load(*want))


@pytest.mark.parametrize("causal", [True, False])
def test_against_64_bits_on_many_tiles(causal):
    """Longer sequences, more items than SMs, walks cut into pieces: against 64 bits on the GPU, one head at a time."""
    gdn = _gdn()
    lens, HQ, HK, D = [1900, 333], 8, 2, 128
    q, k, v, do = _inputs(lens, None, HQ, HK, D, 31)
    c = tuple(t.cuda() for t in (q, k, v, do))
    o, lse, dq, dk, dv = _all(*c, cu_seqlens=U.offsets(lens).cuda(), causal=causal)
    r = {}
    for hk in range(HK):
        part = U.attention(c[0][:, 4 * hk:4 * hk + 4], c[1][:, hk:hk + 1], c[2][:, hk:hk + 1], U.spans(lens), causal, D ** -0.5,
                           c[3][:, 4 * hk:4 * hk + 4])
        for n, t in part.items():
            r.setdefault(n, []).append(t.cpu())
    r = {n: torch.cat(t, 1) for n, t in r.items()}
    _check_fwd(o, lse, r)
    _check_bwd((dq, dk, dv), r)


def test_gradients_against_differences():
    """The gradient along a direction against central differences of a loss, both in 64 bits on the kernels' values: the
    loss is linear in o, whose roundings (2^-8 of each element, independent) bound the difference's error."""
    gdn = _gdn()
    q, k, v, w = _inputs([160], None, 2, 1, 64, 41, q_size=1.0)
    cq, ck, cv, cw = (t.cuda() for t in (q, k, v, w))
    o, lse = gdn.gdn_attention_fwd(cq, ck, cv)
    grads = gdn.gdn_attention_bwd(cw, cq, ck, cv, o, lse)
    g = torch.Generator().manual_seed(5)
    for which, base in enumerate((q, k, v)):
        step = (0.5 * torch.randn(base.shape, generator=g)).to(BF)
        ends = []
        for sign in (1, -1):
            moved = [t.double() for t in (q, k, v)]
            moved[which] = moved[which] + sign * step.double() * 2.0 ** -6
            rows = [(0, 160, 0, 160)]
            ends.append((U.attention(*moved, rows, True, 64 ** -0.5)["o"] * w.double()).sum())
        slope = (ends[0] - ends[1]) / 2.0 ** -5
        got = (grads[which].double().cpu() * step.double()).sum()
        # each gradient element is off by 2^-8 of itself and of its terms at most; along a random direction these add as
        # a root of squares; 4 of them
        r = U.attention(q, k, v, [(0, 160, 0, 160)], True, 64 ** -0.5, w)
        n = ("dq", "dk", "dv")[which]
        err = 2.0 ** -8 * (r[n].abs() + r[n + "_round"] + r[n + "_delta"]) * step.double().abs()
        assert (got - slope).abs() <= 4 * err.square().sum().sqrt() + 1e-3 * slope.abs(), (n, float(got), float(slope))


def test_autograd_entries():
    gdn = _gdn()
    q, k, v, do = (t.cuda() for t in _inputs([90, 41], None, 4, 2, 64, 51))
    cu = U.offsets([90, 41]).cuda()
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    o = gdn.attention(*leaves, cu_seqlens=cu)
    grads = torch.autograd.grad(o, leaves, do)
    want = _all(q, k, v, do, cu_seqlens=cu)
    assert _same_bits([o] + list(grads), [want[0]] + list(want[2:]))
    with pytest.raises(RuntimeError):  # no second derivative
        first = torch.autograd.grad(gdn.attention(*leaves, cu_seqlens=cu).float().sum(), leaves, create_graph=True)
        torch.autograd.grad(sum(t.float().sum() for t in first), leaves)
    # a projection that keeps its input in 8 bits: the input's gradient is that of a plain one, the weight's that of the
    # input's codes
    x = torch.randn(70, 256, device="cuda").to(BF).requires_grad_(True)
    w = torch.randn(96, 256, device="cuda").to(BF).requires_grad_(True)
    dy = torch.randn(70, 96, device="cuda").to(BF)
    y = gdn.linear8(x, w)
    assert torch.equal(y, x @ w.T)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert torch.equal(dx, dy @ w) and torch.equal(dw, dy.T @ gdn.gdn_act8_load(*gdn.gdn_act8_save(x.detach())))
    (dx,) = torch.autograd.grad(gdn.linear8(x, w.detach()), x, dy)
    assert torch.equal(dx, dy @ w)
    # the norm with codes
    x = torch.randn(40, 4, 128, device="cuda").to(BF).requires_grad_(True)
    z, res = (torch.randn(40, 4, 128, device="cuda").to(BF).requires_grad_(True) for _ in range(2))
    w = (1 + 0.1 * torch.randn(128, device="cuda")).requires_grad_(True)
    y, h = gdn.norm_gate(x, w, residual=res, z=z, res_scale=0.5, save8=True)
    dy, dh = torch.randn_like(y), torch.randn_like(h)
    got = torch.autograd.grad((y, h), (x, w, res, z), (dy, dh))
    _, _, h8, hs, z8, zs = gdn.gdn_norm_gate_save8(x.detach(), w.detach(), residual=res.detach(), z=z.detach(), res_scale=0.5)
    dx, dres, dz, dw = gdn.gdn_norm_gate_bwd8(dy, h8, hs, w.detach(), z_codes=z8, z_scale=zs, dh=dh, res_scale=0.5)
    assert all(torch.equal(a, b) for a, b in zip(got, (dx, dw, dres, dz)))
    y, h = gdn.norm_gate(x, w, save8=True)
    assert h is None and torch.autograd.grad(y.float().sum(), x)[0].shape == x.shape


def test_refused_types_and_layouts():
    gdn = _gdn()
    q, k, v, do = (t.cuda() for t in _inputs([32], None, 4, 2, 64, 61))
    lse = torch.zeros(32, 4, device="cuda")
    for bad in (lambda: gdn.gdn_attention_fwd(q.half(), k, v), lambda: gdn.gdn_attention_fwd(q, k.float(), v),
                lambda: gdn.gdn_attention_fwd(q, k, v, cu_seqlens=torch.tensor([0, 32], device="cuda")),
                lambda: gdn.gdn_attention_bwd(do, q, k, v, q, lse.double())):
        with pytest.raises(TypeError):
            bad()
    cu = U.offsets([32]).cuda()
    for bad in (lambda: gdn.gdn_attention_fwd(q[0], k, v), lambda: gdn.gdn_attention_fwd(q, k[:, :, :32], v),
                lambda: gdn.gdn_attention_fwd(q.transpose(0, 1), k, v), lambda: gdn.gdn_attention_fwd(q, k, v[:-1]),
                lambda: gdn.gdn_attention_fwd(q, k, v.cpu()), lambda: gdn.gdn_attention_fwd(q, k[:16], v[:16], cu_seqlens=cu),
                lambda: gdn.gdn_attention_fwd(q, k, v, cu_seqlens_k=cu), lambda: gdn.gdn_attention_fwd(q, k, v, lse=lse[:, :2].contiguous()),
                lambda: gdn.gdn_attention_bwd(do[:, :2], q, k, v, q, lse), lambda: gdn.gdn_act8_load(torch.zeros(3, 256, device="cuda").to(torch.float8_e4m3fn), torch.ones(3, 1, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gdn.gdn_attention_fwd(q[:, :3], k, v),  # 3 heads over 2
                lambda: gdn.gdn_attention_fwd(*(torch.zeros(8, 2, 96, device="cuda", dtype=BF),) * 3),
                lambda: gdn.gdn_attention_fwd(torch.zeros(32 * 260 + 8, device="cuda", dtype=BF).as_strided((32, 4, 64), (260, 64, 1)), k, v),
                lambda: gdn.gdn_norm_gate_save8(torch.zeros(3, 130, device="cuda", dtype=BF), torch.ones(130, device="cuda"))):
        with pytest.raises(gdn.GDNError):
            bad()


@pytest.mark.parametrize("D", [128, 64])
def test_a_wait_that_runs_out(D):
    """The testing switch makes a bounded wait of every block run out: the call reports it and ends, and the next one is
    right."""
    gdn = _gdn()
    q, k, v, do = (t.cuda() for t in _inputs([700, 133], None, 4, 2, D, 71))
    cu = U.offsets([700, 133]).cuda()
    want = _all(q, k, v, do, cu_seqlens=cu)
    for call in (lambda st: gdn.gdn_attention_fwd(q, k, v, cu_seqlens=cu, dev_status=st),
                 lambda st: gdn.gdn_attention_bwd(do, q, k, v, *want[:2], cu_seqlens=cu, dev_status=st)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        prev = gdn.testing_force_wait_expiry(True)
        try:
            call(st)
            torch.cuda.synchronize()
        finally:
            gdn.testing_force_wait_expiry(prev)
        assert int(st) & gdn.DEV_WAIT_TIMEOUT and not int(st) & gdn.DEV_DRAIN_TIMEOUT
        st.zero_()
        assert _same_bits(_all(q, k, v, do, cu_seqlens=cu, dev_status=st), want) and int(st) == 0


def test_gradients_that_arrive_at_an_odd_address():
    """The gradient of a piece of a concatenation is a view that starts where the piece does."""
    gdn = _gdn()
    g = torch.Generator().manual_seed(5)
    T, H, D = 37, 2, 64

    def leaf(*shape):
        return torch.randn(*shape, generator=g).to(BF).cuda().requires_grad_()

    q, k, v, x, r, z = (leaf(T, H, D) for _ in range(6))
    w = (1.0 + 0.1 * torch.randn(D, generator=g)).cuda().requires_grad_()
    up = torch.randn(3 * T * H * D + 3, generator=g).to(BF).cuda()
    leaves = (q, k, v, x, r, z, w)
    out = [gdn.attention(q, k, v), *gdn.norm_gate(x, w, residual=r, z=z, save8=True)]
    n = out[0].numel()
    one = torch.zeros(1, dtype=BF, device="cuda")
    odd = torch.cat([t for o in out for t in (one, o.flatten())])
    got = torch.autograd.grad(odd, leaves, up, retain_graph=True)
    want = torch.autograd.grad(out, leaves, [up[i * (n + 1) + 1:(i + 1) * (n + 1)].clone().view(T, H, D) for i in range(3)])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("order", ["random", "grow", "fall"])
@pytest.mark.parametrize("D,causal", [(128, True), (64, True), (64, False)])
@pytest.mark.parametrize("power,scale", [(8, 1.0), (17, 1.0), (23, 1.0), (24, 1.0), (25, 3.0), (31, 1.0), (60, 0.5), (100, 1.0), (119, 3.0)])
def test_logits_of_any_size(power, scale, D, causal, order):
    """Logits of 2^power times whole numbers, exact in bf16 and in the products, up to where scale q k itself passes fp32:
    the largest of a row take all the weight.  o is a mean of some values.  Its weights are 2^(c S - c m) with c m rounded,
    the same number near 1 for all of them, which enters the product in bf16, off by 2^-8 of itself, and the sum l before
    that rounding: 2^-8 of the mean's terms, and 2^-8 of the mean for the output's rounding.  The factors of lse are off
    by 2^-24 each, four of them."""
    gdn = _gdn()
    T = 300
    g = torch.Generator().manual_seed(power)
    n = torch.randint(-120, 121, (T,), generator=g).double()
    n = n if order == "random" else n.sort(descending=order == "fall")[0]
    q, k = torch.zeros(T, 1, D), torch.zeros(T, 1, D)
    q[:, 0, 3], k[:, 0, 3] = 2.0 ** power, n.float()
    v = torch.randn(T, 1, D, generator=g).to(BF)
    o, lse = gdn.gdn_attention_fwd(q.to(BF).cuda(), k.to(BF).cuda(), v.cuda(), causal=causal, scale=scale)
    s = (n * 2.0 ** power * scale).expand(T, T)
    if causal:
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool).triu(1), -math.inf)
    p = (s == s.amax(-1, keepdim=True)).double()
    p /= p.sum(-1, keepdim=True)
    want, mag = p @ v[:, 0].double(), p @ v[:, 0].double().abs()
    _near(o[:, 0], want, 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -20) * mag, "o")
    ref = torch.logsumexp(s, -1)
    ref = torch.where(ref.abs() > torch.finfo(torch.float32).max, ref.sign() * math.inf, ref)
    _near(lse[:, 0], ref, 2.0 ** -22 * ref.abs() + 2.0 ** -20, "lse")


def _few(N, at):
    lens = [0] * N
    for n, m in at.items():
        lens[n] = m
    return lens


@pytest.mark.parametrize("lens,lens_k,HQ,HK,D", [
    (_few(600, {3: 200, 4: 7, 300: 60, 599: 23}), None, 4, 1, 128),       # walks that are cut, places by rows
    (_few(1024, {0: 37}), None, 2, 2, 64),
    (_few(300, {5: 400, 200: 130}), _few(300, {5: 100, 200: 150}), 2, 1, 128),  # rows and keys find theirs in different ways
    (_few(300, {5: 30, 200: 13}), _few(300, {5: 500, 200: 150, 250: 9}), 2, 1, 64),
])
@pytest.mark.parametrize("causal", [True, False])
def test_mostly_empty_sequences(lens, lens_k, HQ, HK, D, causal):
    """Offsets of many empty sequences, as a padded batch has them: a workspace as large as it has to be, nothing behind it
    written."""
    gdn = _gdn()
    q, k, v, do = _inputs(lens, lens_k, HQ, HK, D, 3)
    cu, cu_k = U.offsets(lens).cuda(), None if lens_k is None else U.offsets(lens_k).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(cu_seqlens=cu, cu_seqlens_k=cu_k, causal=causal, dev_status=status)
    c = [t.cuda() for t in (q, k, v)]
    o, lse = gdn.gdn_attention_fwd(*c, **args)
    need = gdn.attention_bwd_workspace_size(len(lens), sum(lens), len(k), HQ, HK, D)
    buffer = torch.full((need + (1 << 20),), 0x5a, dtype=torch.uint8, device="cuda")
    grads = gdn.gdn_attention_bwd(do.cuda(), *c, o, lse, workspace=buffer[:need], **args)
    assert int(status) == 0 and bool((buffer[need:] == 0x5a).all())
    r = U.attention(q, k, v, U.spans(lens, lens_k), causal, D ** -0.5, do)
    _check_fwd(o, lse, r)
    _check_bwd(grads, r)


def test_autograd_reports_bad_offsets():
    gdn = _gdn()
    q, k, v, do = (t.cuda() for t in _inputs([300], None, 2, 1, 64, 9))
    leaves = [t.requires_grad_() for t in (q, k, v)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = gdn.attention(*leaves, cu_seqlens=torch.tensor([0, 100, 400], dtype=torch.int32, device="cuda"), dev_status=st)
    assert int(st) == gdn.DEV_BAD_CU_SEQLENS
    st.zero_()  # between the directions: the caller's to do
    torch.autograd.grad(o, leaves, do)
    assert int(st) == gdn.DEV_BAD_CU_SEQLENS
    st.zero_()
    torch.autograd.grad(gdn.attention(*leaves, cu_seqlens=U.offsets([100, 200]).cuda(), dev_status=st), leaves, do)
    assert int(st) == 0


def _odd(t):
    """The same values two bytes past a boundary."""
    o = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    return o.copy_(t)


@pytest.mark.parametrize("kind,res", [("silu", True), (None, False), ("sigmoid", False)])
@pytest.mark.parametrize("layout", ["odd", "stride", "both"])
def test_norm_with_codes_of_inputs_that_lie_anywhere(kind, res, layout):
    """What norm_gate takes without codes it takes with them: the same results as of aligned copies."""
    gdn = _gdn()
    g = torch.Generator().manual_seed(8)
    x, r, z, dy, dh = (torch.randn(37, 4, 96, generator=g).to(BF).cuda() for _ in range(5))
    w = (1 + 0.1 * torch.randn(96, generator=g)).cuda()
    args = dict(activation=kind or "silu", res_scale=0.5 if res else 1.0)

    def run(x, r, z, save8=True):
        leaves = [x.detach().requires_grad_(), w.detach().requires_grad_()] + [t.detach().requires_grad_() for t, on in ((r, res), (z, kind)) if on]
        y, h = gdn.norm_gate(leaves[0], leaves[1], residual=leaves[2] if res else None, z=leaves[-1] if kind else None, save8=save8, **args)
        grads = torch.autograd.grad((y, h) if res else y, leaves, (dy, dh) if res else dy)
        return [y.detach(), *grads] + ([h.detach()] if res else [])

    want = run(x, r, z)
    if layout != "stride":
        x, r = _odd(x), _odd(r)
    if layout != "odd":  # rows of 4 x 96 + 4
        wide = torch.zeros(37, 4 * 96 + 4, dtype=BF, device="cuda")
        z = wide[:, 4 if layout == "both" else 0:][:, :4 * 96].unflatten(1, (4, 96)).copy_(z)
    else:
        z = _odd(z)
    assert all(torch.equal(a, b) for a, b in zip(run(x, r, z), want))
    assert torch.equal(run(x, r, z, False)[0], want[0])


@pytest.mark.parametrize("D", [1, 100, 130, 16392])
@pytest.mark.parametrize("kind,res", [("silu", True), (None, False)])
def test_norm_with_codes_of_any_width(D, kind, res):
    """Widths that only the norm without codes takes: its results, and its gradients at the values of the codes."""
    gdn = _gdn()
    g = torch.Generator().manual_seed(D)
    x, r, z, dy, dh = (torch.randn(5, 2, D, generator=g).to(BF).cuda() for _ in range(5))
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    leaves = [t.requires_grad_() for t in (x, w, *([r] if res else []), *([z] if kind else []))]
    args = dict(residual=r if res else None, z=z if kind else None)
    y, h = gdn.norm_gate(x, w, save8=True, **args)
    want, stream = gdn.gdn_norm_gate(x.detach(), w.detach(), **{n: None if t is None else t.detach() for n, t in args.items()})
    assert torch.equal(y, want) and (h is None if not res else torch.equal(h, stream))
    values = lambda t: gdn.gdn_act8_load(*gdn.gdn_act8_save(t.detach()))  # noqa: E731
    dx, dres, dz, dw = gdn.gdn_norm_gate_bwd(dy, values(h if res else x), w.detach(), z=values(z) if kind else None, dh=dh if res else None)
    got = torch.autograd.grad((y, h) if res else y, leaves, (dy, dh) if res else dy)
    assert all(torch.equal(a, b) for a, b in zip(got, [dx, dw] + ([dres] if res else []) + ([dz] if kind else [])))


def test_linear8_of_any_strides():
    gdn = _gdn()
    g = torch.Generator().manual_seed(9)
    w = torch.randn(40, 96, generator=g).to(BF).cuda().requires_grad_()
    base = torch.randn(6, 7, 96, generator=g).to(BF).cuda()
    for x in (base.transpose(0, 1), base.transpose(1, 2).contiguous().transpose(1, 2), _odd(base), base[0].T.contiguous().T, base[0, 0],
              base[:, :1].expand(6, 7, 96), base[:0]):
        x = x.detach().requires_grad_()
        y = gdn.linear8(x, w)
        dy = torch.randn(y.shape, generator=g).to(BF).cuda()
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        rows, d = x.detach().reshape(-1, 96).contiguous(), dy.reshape(-1, 40)
        assert torch.equal(y, x @ w.T) and dx.shape == x.shape and torch.equal(dx, dy @ w.detach())
        assert torch.equal(dw, d.T @ gdn.gdn_act8_load(*gdn.gdn_act8_save(rows)))


def test_walks_of_more_than_a_second():
    """304 key tiles, one kv head, 1024 query heads: a walk has 2 million steps of 128 rows, whose 128 x 128 exponentials
    take 1024 cycles a step at least (16 a cycle), so 2.1e9 cycles: no wait takes that for a partner that is gone."""
    gdn = _gdn()
    T, HQ, keys, D = 1984 * 128, 1024, 304 * 128, 64
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.zeros(T, HQ, D, dtype=BF, device="cuda")  # o and its gradient too
    k, v = (torch.ones(keys, 1, D, dtype=BF, device="cuda") for _ in range(2))
    status = ints(0)
    dq, dk, dv = gdn.gdn_attention_bwd(q, q, k, v, q, torch.zeros(T, HQ, device="cuda"), cu_seqlens=ints(0, T),
                                       cu_seqlens_k=ints(0, keys), causal=False, dev_status=status)
    assert int(status) == 0
    assert not dk.any() and not dv.any() and all(not t.any() for t in dq.split(4096))


def test_sequences_that_overlap_are_left_out():
    """Offsets that go back and forth: of the sequences that name the same rows the first has them, and the call does no
    more work than the rows are, in every chunk of 32 sequences."""
    gdn = _gdn()
    T = 300
    q, k, v, do = (t.cuda() for t in _inputs([T], [2 * T], 2, 1, 64, 10))
    for N in (3, 501):
        cu = torch.tensor([0, T] * (N // 2 + 1), dtype=torch.int32, device="cuda")
        cu_k = torch.tensor([0, T] + [T, 2 * T] * (N // 2), dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        o, lse = gdn.gdn_attention_fwd(q, k, v, cu_seqlens=cu, cu_seqlens_k=cu_k, causal=False, dev_status=st)
        assert int(st) == gdn.DEV_BAD_CU_SEQLENS
        assert _same_bits((o, lse), gdn.gdn_attention_fwd(q, k[:T], v[:T], causal=False))
        st.zero_()
        gdn.gdn_attention_bwd(do, q, k, v, o, lse, cu_seqlens=cu, cu_seqlens_k=cu_k, causal=False, dev_status=st)
        assert int(st) == gdn.DEV_BAD_CU_SEQLENS


@pytest.mark.parametrize("causal", [True, False])
def test_as_many_sequences_as_there_may_be(causal):
    g = torch.Generator().manual_seed(12)
    full = torch.randperm(65535, generator=g)[:60].tolist() + [65534]
    lens, lens_k = [0] * 65535, [0] * 65535
    for n, m, d in zip(full, torch.randint(1, 160, (61,), generator=g).tolist(), torch.randint(-30, 60, (61,), generator=g).tolist()):
        lens[n], lens_k[n] = m, max(0, m + d)
    _run(lens, None, 2, 1, 128, causal, 13)
    _run(lens, lens_k, 2, 2, 64, causal, 14)


@pytest.mark.parametrize("HK", [15, 1])
def test_as_many_heads_as_there_may_be(HK):
    """65535 query heads, against 64 bits for all of them at once, on the GPU."""
    gdn = _gdn()
    T, HQ, D = 5, 65535, 64
    q, k, v, do = (t.cuda() for t in _inputs([T], None, HQ, HK, D, 17))
    o, lse, *grads = _all(q, k, v, do)
    r, scale = {}, D ** -0.5
    q, do = (t.double().view(T, HK, HQ // HK, D) for t in (q, do))
    k, v = k.double(), v.double()
    hidden = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)

    def pairs(a, b):
        return torch.einsum("ihgd,jhd->hgij", a, b)

    def to_rows(p, b):
        return torch.einsum("hgij,jhd->ihgd", p, b)

    def to_keys(p, a):
        return torch.einsum("hgij,ihgd->jhd", p, a)

    s = (pairs(q, k) * scale).masked_fill(hidden, -math.inf)
    size = 1 + (pairs(q.abs(), k.abs()) * scale).masked_fill(hidden, 0).amax(-1, keepdim=True)
    p = s.softmax(-1)
    r["o"], r["o_mag"], r["lse"], r["lse_mag"] = to_rows(p, v), to_rows(p, v.abs()), s.logsumexp(-1), size[..., 0]
    delta = (do * r["o"]).sum(-1).permute(1, 2, 0)[..., None]
    terms = (do * r["o"]).abs().sum(-1).permute(1, 2, 0)[..., None]
    ds, mag = p * (pairs(do, v) - delta), p * (pairs(do.abs(), v.abs()) + terms) * size
    for n, ways in (("", (scale * ds, p)), ("_round", (scale * ds.abs(), p)), ("_fp32", (scale * mag, p * size)), ("_delta", (scale * p * terms, p))):
        f = (lambda t: t) if n == "" else torch.abs
        r["dq" + n], r["dk" + n], r["dv" + n] = to_rows(ways[0], f(k)), to_keys(ways[0], f(q)), to_keys(ways[1], f(do))
    rows = lambda t: t.reshape(T, HQ, D).cpu()  # noqa: E731
    heads = lambda t: t.permute(2, 0, 1).reshape(T, HQ).cpu()  # noqa: E731
    r = {n: heads(t) if n.startswith("lse") else rows(t) if n[0] == "o" or n.startswith("dq") else t.cpu() for n, t in r.items()}
    _check_fwd(o, lse, r)
    _check_bwd(grads, r)
