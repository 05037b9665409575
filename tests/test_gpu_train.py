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
