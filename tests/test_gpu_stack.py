"""The operators around the recurrence on the GPU against plain 64-bit implementations (tests/stack_util.py).

Tolerances, from the roundings: a bf16 output is one rounding of an fp32 result, 2^-9 relative, and the fp32 result is
off by some 2^-21 of the terms that were added, so 2^-8 of the value plus 2^-18 of the largest term.  fp32 sums over
rows: 2^-19 of the sum of magnitudes.  Attention: p is rounded to 11 bits (2^-12 each, at most 2^-11 of
sum p |v| with the fp32 errors of the logits) and o to bf16.  Codes, scales and whole numbers: equal."""
import math

import numpy as np
import pytest
import torch

import stack_util as U

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_chunked_chunk_gb300 import build
    build.build()


def _gdn():
    import gated_deltanet_chunked_chunk_gb300 as gdn
    return gdn


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _close_bf16(got, ref, extra=0.0, what=""):
    got = U.f64(got)
    tol = 2.0 ** -8 * np.abs(ref) + extra + 1e-37
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(np.abs(got - ref) - tol):.3e}"


# ------------------------------------------------------------------- norms
@pytest.mark.parametrize("shape", [(1, 128), (257, 2, 128), (33, 4, 64), (5, 3, 96), (130, 256), (9, 512), (7, 1024), (5, 2048),
                                   (3, 4096), (3, 8192), (2, 16384), (2, 16392), (4, 1), (6, 7), (3, 1001), (2, 3, 130)])
@pytest.mark.parametrize("kind,res", [(None, False), ("silu", True), ("sigmoid", False)])
def test_norm_gate_and_gradients(shape, kind, res):
    gdn, g = _gdn(), _gen(sum(shape))
    x = (2 * torch.randn(shape, generator=g)).to(BF)
    w = 1 + 0.1 * torch.randn(shape[-1], generator=g)
    z = torch.randn(shape, generator=g).to(BF) if kind else None
    r = torch.randn(shape, generator=g).to(BF) if res else None
    dy, dh = torch.randn(shape, generator=g).to(BF), torch.randn(shape, generator=g).to(BF) if res else None
    c = lambda t: None if t is None else t.cuda()
    y, h = gdn.gdn_norm_gate(c(x), c(w), residual=c(r), z=c(z), activation=kind, res_scale=0.5 if res else 1.0)
    ry, rh = U.norm_fwd(U.f64(x), U.f64(w), U.f64(r), U.f64(z), kind, res_scale=0.5 if res else 1.0)
    _close_bf16(y, ry, what="y")
    if res:
        _close_bf16(h, rh, 2.0 ** -18 * np.abs(rh).max(), what="h")
    else:
        assert h is None
    hb = x if h is None else h.cpu()
    dx, dres, dz, dw = gdn.gdn_norm_gate_bwd(c(dy), c(hb), c(w), z=c(z), dh=c(dh), activation=kind,
                                             res_scale=0.5 if res else 1.0)
    h64 = U.f64(hb)
    rx, rr, rz, rw = U.norm_bwd(U.f64(dy), h64, U.f64(w), U.f64(z), U.f64(dh), kind, res_scale=0.5 if res else 1.0)
    rstd = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + 1e-6)
    terms = rstd * np.abs(U.f64(dy)).max(-1, keepdims=True) * 4 + (2.0 if res else 0.0)
    _close_bf16(dx, rx, 2.0 ** -18 * terms, what="dx")
    if res:
        _close_bf16(dres, rr, 2.0 ** -18 * terms, what="dresidual")
    if kind:
        _close_bf16(dz, rz, 2.0 ** -18 * np.abs(U.f64(dy) * h64 * rstd), what="dz")
    n = h64 * rstd
    mags = np.abs(U.f64(dy) * n * (1.0 if kind is None else U.act(U.f64(z), kind)[0])).reshape(-1, shape[-1]).sum(0)
    assert (np.abs(U.f64(dw) - rw) <= 2.0 ** -19 * mags + 1e-30).all()


def test_norm_gate_of_a_packed_projection_in_place_and_misaligned():
    gdn, g = _gdn(), _gen(3)
    T, H, D = 37, 4, 128
    wide = torch.randn(T, 3 * H * D + 8, generator=g).to(BF).cuda()
    z = wide[:, H * D:2 * H * D].view(T, H, D)
    assert not z.is_contiguous()
    x = torch.randn(T, H, D, generator=g).to(BF).cuda()
    w = torch.rand(D, generator=g).cuda() + 0.5
    y, _ = gdn.gdn_norm_gate(x, w, z=z)
    y2, _ = gdn.gdn_norm_gate(x, w, z=z.contiguous())
    assert torch.equal(y, y2)
    a = gdn.gdn_norm_gate_bwd(x, y, w, z=z)
    b = gdn.gdn_norm_gate_bwd(x, y, w, z=z.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)
    # the same values from buffers that are only 2-byte aligned (the element loop): equal up to fp32 order
    buf = torch.empty(x.numel() + 1, dtype=BF, device="cuda")
    odd = buf[1:].view(T, H, D)
    odd.copy_(x)
    y3, _ = gdn.gdn_norm_gate(odd, w, z=z)
    ry, _ = U.norm_fwd(U.f64(x), U.f64(w), None, U.f64(z))
    _close_bf16(y3, ry, what="misaligned")
    # in place: y over x, h over the residual
    r = torch.randn(T, H, D, generator=g).to(BF).cuda()
    y4, h4 = gdn.gdn_norm_gate(x, w, residual=r, res_scale=0.25)
    xi, ri = x.clone(), r.clone()
    y5, h5 = gdn.gdn_norm_gate(xi, w, residual=ri, res_scale=0.25, y=xi, h=ri)
    assert y5.data_ptr() == xi.data_ptr() and torch.equal(y4, y5) and torch.equal(h4, h5)


def test_norm_gate_extremes():
    gdn = _gdn()
    D = 128
    x = torch.zeros(4, D)
    x[1, 5] = 1e30   # one large element: the others vanish, the row keeps its norm
    x[2] = 1e-20     # far below eps
    x[3] = 3.0
    z = torch.zeros(4, D)
    z[3, 0], z[3, 1] = 200.0, -200.0
    x, z = x.to(BF), z.to(BF)
    w = torch.ones(D)
    y, _ = gdn.gdn_norm_gate(x[:1].cuda(), w.cuda())
    assert (y == 0).all()
    y, _ = gdn.gdn_norm_gate(x[2:].cuda(), w.cuda(), z=z[2:].cuda())
    ry, _ = U.norm_fwd(U.f64(x[2:]), U.f64(w), None, U.f64(z[2:]))
    _close_bf16(y, ry, 1e-30)
    nan = x[3:].clone()
    nan[0, 7] = float("nan")
    y, _ = gdn.gdn_norm_gate(torch.cat([x[3:], nan]).cuda(), w.cuda())
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1]).all()
    y, h = gdn.gdn_norm_gate(torch.empty(0, D, dtype=BF, device="cuda"), w.cuda())
    assert y.shape == (0, D) and h is None
    e = torch.empty(0, D, dtype=BF, device="cuda")
    dx, _, _, dw = gdn.gdn_norm_gate_bwd(e, e, w.cuda())
    assert dx.shape == (0, D) and (dw == 0).all()


def test_norm_gate_autograd_against_differences_and_repeats():
    """The gradient against central differences of the 64-bit forward, along random directions, and bit for bit twice."""
    gdn, g = _gdn(), _gen(11)
    T, D = 6, 64
    x, r, z = (torch.randn(T, D, generator=g).to(BF) for _ in range(3))
    w = 1 + 0.1 * torch.randn(D, generator=g)
    cy, ch = torch.randn(T, D, generator=g).to(BF), torch.randn(T, D, generator=g).to(BF)
    leaves = [t.cuda().requires_grad_() for t in (x, w, r, z)]
    y, h = gdn.norm_gate(leaves[0], leaves[1], residual=leaves[2], z=leaves[3], res_scale=0.5)
    grads = torch.autograd.grad([y, h], leaves, [cy.cuda(), ch.cuda()])
    again = torch.autograd.grad(gdn.norm_gate(leaves[0], leaves[1], residual=leaves[2], z=leaves[3], res_scale=0.5), leaves,
                                [cy.cuda(), ch.cuda()])
    assert all(torch.equal(a, b) for a, b in zip(grads, again))

    def loss(x, w, r, z):
        y, h = U.norm_fwd(x, w, r, z, "silu", res_scale=0.5)
        return (y * U.f64(cy)).sum() + (h * U.f64(ch)).sum()

    base = [U.f64(t) for t in (x, w, r, z)]
    for i in range(4):
        for k in range(3):
            d = np.random.RandomState(10 * i + k).randn(*base[i].shape)
            step = 1e-5
            up, dn = list(base), list(base)
            up[i], dn[i] = base[i] + step * d, base[i] - step * d
            num = (loss(*up) - loss(*dn)) / (2 * step)
            got = (U.f64(grads[i]) * d).sum()
            # bf16 gradients of a stream that the forward stored in bf16: 2^-8 of each term, added at random
            tol = 2.0 ** -8 * 4 * np.sqrt(((U.f64(grads[i]) * d) ** 2).sum()) + 2.0 ** -8 * np.abs(U.f64(grads[i])).max()
            assert abs(num - got) <= tol, (i, k, num, got, tol)


# ------------------------------------------------------------------ rotary
@pytest.mark.parametrize("T,HQ,HK,D,rot", [(1, 1, 1, 64, 64), (3, 32, 4, 128, 32), (257, 8, 2, 128, 128), (5000, 4, 1, 64, 16),
                                           (19, 3, 1, 256, 128), (7, 2, 2, 80, 20), (11, 2, 0, 10, 6), (40, 16, 16, 128, 64),
                                           (2, 1, 1, 2, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_and_inverse(T, HQ, HK, D, rot, interleaved):
    gdn, g = _gdn(), _gen(T + D)
    q = torch.randn(T, HQ, D, generator=g).to(BF)
    k = torch.randn(T, HK, D, generator=g).to(BF) if HK else None
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0] = 2147483647 if T > 1 else 0
    pos[-1] = -5 if T > 2 else pos[-1]
    inv, att = gdn.rope_frequencies(rot, scaling="yarn", factor=4.0)
    att = 1.25
    c = lambda t: None if t is None else t.cuda()
    for inverse in (False, True):
        qo, ko = gdn.gdn_rope(c(q), c(k), c(pos), c(inv), interleaved=interleaved, attention_factor=att, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            if x is None:
                assert y is None
                continue
            ref = U.rope(U.f64(x), pos.numpy(), inv.numpy(), interleaved, att, inverse)
            _close_bf16(y, ref, 2.0 ** -18 * np.abs(U.f64(x)).max(), what="rope")
            assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


def test_rope_views_in_place_and_gradient():
    gdn, g = _gdn(), _gen(5)
    T, HQ, HK, D = 70, 8, 2, 128
    packed = torch.randn(T, (HQ + 2 * HK) * D, generator=g).to(BF).cuda()
    q, k = packed[:, :HQ * D].view(T, HQ, D), packed[:, HQ * D:(HQ + HK) * D].view(T, HK, D)
    pos = torch.arange(T, dtype=torch.int32).cuda() * 37
    inv, _ = gdn.rope_frequencies(D, device="cuda")
    a = gdn.gdn_rope(q, k, pos, inv)
    qc, kc = q.contiguous(), k.contiguous()
    b = gdn.gdn_rope(qc, kc, pos, inv, q_out=qc, k_out=kc)
    assert b[0].data_ptr() == qc.data_ptr() and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # an odd element offset takes the element loop: the same formula in fp32, at most a rounding apart
    buf = torch.empty(T * HQ * D + 1, dtype=BF, device="cuda")
    buf[1:].copy_(q.reshape(-1))
    odd, _ = gdn.gdn_rope(buf[1:].view(T, HQ, D), None, pos, inv)
    _close_bf16(odd, U.rope(U.f64(q), pos.cpu().numpy(), inv.cpu().numpy(), False), 2.0 ** -16)
    ql, kl = q.detach().clone().requires_grad_(), k.detach().clone().requires_grad_()
    co = torch.randn(T, HQ, D, generator=g).to(BF).cuda(), torch.randn(T, HK, D, generator=g).to(BF).cuda()
    out = gdn.rotary_embedding(ql, kl, pos, inv, attention_factor=1.5)
    dq, dk = torch.autograd.grad(out, (ql, kl), co)
    # <R x, c> = <x, R^T c>, and the difference quotient of a linear map is the map itself
    for x, d, cc in ((q, dq, co[0]), (k, dk, co[1])):
        lhs = U.rope(U.f64(x), pos.cpu().numpy(), inv.cpu().numpy(), False, 1.5) * U.f64(cc)
        assert abs(lhs.sum() - (U.f64(x) * U.f64(d)).sum()) <= 4 * 2.0 ** -8 * np.sqrt((lhs ** 2).sum() + (U.f64(x) * U.f64(d)).var() * d.numel())
    e = gdn.gdn_rope(q[:0], k[:0], pos[:0], inv)
    assert e[0].shape == (0, HQ, D)


# -------------------------------------------------------------------- plan
def _plan_case(N, cached_hi, new_hi, bs, seed, extra=4):
    r = np.random.RandomState(seed)
    cached = r.randint(0, cached_hi + 1, N).tolist()
    new = r.randint(0, new_hi + 1, N).tolist()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
    width = max(1, max(-(-(c + m) // bs) for c, m in zip(cached, new))) + 1
    ids = r.permutation(sum(-(-(c + m) // bs) for c, m in zip(cached, new)) + extra).tolist()
    table = [[-1] * width for _ in range(N)]
    for n, c in enumerate(cached):
        for p in range(-(-c // bs)):
            table[n][p] = ids.pop()
    return cached, cu, table, ids, bs


def _run_plan(case, left=None, width=None):
    gdn = _gdn()
    cached, cu, table, ids, bs = case
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    left = len(ids) if left is None else left
    t = i(table)
    if width is not None:
        t = t[:, :width].contiguous()
        table = [row[:width] for row in table]
    st = i([0])
    free = i(ids) if ids else torch.empty(0, dtype=torch.int32, device="cuda")
    got = gdn.gdn_paged_plan(i(cached), i(cu), t, free, i([left]), bs, cu[-1], dev_status=st)
    ref = U.plan(cached, cu, table, ids, left, bs, cu[-1])
    return t, got, ref, int(st.item())


@pytest.mark.parametrize("N,cached_hi,new_hi,bs", [(1, 0, 1, 16), (1, 300, 5000, 64), (7, 65, 1, 64), (300, 200, 3, 16), (1024, 70, 9, 32),
                                                   (1025, 5, 2, 128), (3000, 40, 1, 16), (5, 100, 2000, 48)])
def test_plan(N, cached_hi, new_hi, bs):
    case = _plan_case(N, cached_hi, new_hi, bs, N)
    t, got, ref, st = _run_plan(case)
    assert st == 0
    assert t.cpu().tolist() == ref[0]
    for a, b in zip(got, (ref[1], ref[2], ref[3], [ref[4]])):
        assert a.cpu().tolist() == b
    # again on the table that now has the pages: nothing changes
    t2, got2, _, _ = _run_plan((case[0], case[1], t.cpu().tolist(), case[3], bs))
    assert torch.equal(t, t2) and all(torch.equal(a, b) for a, b in zip(got, got2))


def test_plan_without_enough_pages_or_room():
    gdn = _gdn()
    case = _plan_case(40, 60, 50, 16, 3)
    t, got, ref, st = _run_plan(case, left=5)
    assert st == gdn.DEV_NO_PAGE and ref[5]
    assert t.cpu().tolist() == ref[0] and got[1].cpu().tolist() == ref[2] and int(got[3]) == 0
    t, got, ref, st = _run_plan(case, width=3)
    assert st == gdn.DEV_NO_PAGE and got[1].cpu().tolist() == ref[2] and got[2].cpu().tolist() == ref[3]
    assert t.cpu().tolist() == ref[0]


def test_plan_bad_offsets_and_empty():
    gdn = _gdn()
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    st = i([0])
    t = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    # request 1 runs backwards; the tokens that no request has get slot -1
    seq, slots, pos, left = gdn.gdn_paged_plan(i([0, 3, 0]), i([0, 2, 1, 4]), t, i([5, 6, 7, 8]), i([4]), 4, 4, dev_status=st)
    assert int(st) == gdn.DEV_BAD_CU_SEQLENS and seq.tolist() == [2, 3, 3]
    assert all(s == -1 or 0 <= s < 9 * 4 for s in slots.tolist())
    st.zero_()
    seq, slots, pos, left = gdn.gdn_paged_plan(i([-4]), i([0, 1]), t[:1], i([5]), i([1]), 4, 1, dev_status=st)
    assert int(st) == gdn.DEV_BAD_CU_SEQLENS and slots.tolist() == [-1]
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    seq, slots, pos, left = gdn.gdn_paged_plan(e, i([0]), t[:0], i([5]), i([1]), 4, 2)
    assert seq.numel() == 0 and slots.tolist() == [-1, -1] and left.tolist() == [1]
    seq, slots, pos, left = gdn.gdn_paged_plan(i([3]), i([0, 0]), t[:1], i([5]), i([9]), 4, 0)
    assert seq.tolist() == [3] and slots.numel() == 0 and left.tolist() == [1]  # num_free beyond the list counts as its length


# ------------------------------------------------------------------ append
def _same_cache(codes, scale, ref):
    got = U.f64(codes.float())
    assert np.array_equal(np.isnan(got), np.isnan(ref[0])) and np.array_equal(np.nan_to_num(got), np.nan_to_num(ref[0]))
    assert np.array_equal(U.f64(scale), ref[1])


@pytest.mark.parametrize("HK,D,bs,counts,offs", [
    (1, 64, 16, [1], [0]), (2, 128, 64, [1, 1, 1, 1], [0, 5, 63, 17]), (4, 128, 64, [200, 64, 3], [30, 0, 61]),
    (3, 64, 16, [1, 40, 2, 16], [15, 9, 14, 0]), (1, 128, 128, [300], [100]), (2, 72, 8, [20, 5], [3, 0]), (2, 10, 5, [9, 1], [1, 4])])
@pytest.mark.parametrize("packed", [False, True])
def test_append(HK, D, bs, counts, offs, packed):
    gdn, g = _gdn(), _gen(D + bs)
    T, need = sum(counts), [-(-(o + c) // bs) for o, c in zip(offs, counts)]
    P = sum(need) + 2
    ids = torch.randperm(P, generator=g).tolist()
    slots, at = [], 0
    for o, c, m in zip(offs, counts, need):
        pages = ids[at:at + m]
        at += m
        slots += [pages[(o + i) // bs] * bs + (o + i) % bs for i in range(c)]
    slots.insert(0, -1)  # a token without a place (a page's own tokens must follow one another)
    T += 1
    kc, ks = U.make_cache(P, HK, bs, D, g)
    vc, vs = U.make_cache(P, HK, bs, D, g)
    wide = torch.randn(T, 2 * HK * D, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))
    wide = wide.to(BF)
    k, v = (wide[:, :HK * D].view(T, HK, D), wide[:, HK * D:].view(T, HK, D))
    if not packed:
        k, v = k.contiguous(), v.contiguous()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    wd = wide.cuda()
    kd, vd = (wd[:, :HK * D].view(T, HK, D), wd[:, HK * D:].view(T, HK, D)) if packed else (k.cuda(), v.cuda())
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    for _ in range(2):  # the second time the same tokens go to the same places
        gdn.gdn_kv8_append(kd, vd, dev[0], dev[1], dev[2], dev[3], sl, dev_status=st)
        assert int(st) == 0
        _same_cache(dev[0], dev[2], U.append(U.f64(k), U.f64(kc.float()), U.f64(ks), slots))
        _same_cache(dev[1], dev[3], U.append(U.f64(v), U.f64(vc.float()), U.f64(vs), slots))


def test_append_values_at_the_edges():
    """Zeros, infinities, NaN, values on the border of an exponent, growth of a page's scale by much, tiny values."""
    gdn = _gdn()
    bs, D, P = 16, 64, 6
    kc, ks = U.make_cache(P, 1, bs, D, _gen(1))
    rows = torch.zeros(8, 1, D)
    rows[1] = 448.0
    rows[2] = 450.0  # the next bf16
    rows[3, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 2.0])
    rows[4] = 1e30
    rows[5] = 1e-30
    rows[6] = torch.linspace(-1, 1, D)
    rows[7, 0, 0] = float("nan")
    x = rows.to(BF)
    slots = [0 * bs, 1 * bs, 2 * bs, 3 * bs, 4 * bs + 7, 5 * bs]
    dev = [t.cuda() for t in (kc, kc.clone(), ks, ks.clone())]
    ref = U.f64(kc.float()), U.f64(ks)
    for rows, at in ((x[:6], slots), (x[6:], [0 * bs + 1, 1 * bs + 1])):  # the second call adds to pages of the first
        gdn.gdn_kv8_append(rows.cuda(), rows.cuda(), dev[0], dev[1], dev[2], dev[3], torch.tensor(at, dtype=torch.int32, device="cuda"))
        ref = U.append(U.f64(rows), ref[0], ref[1], at)
        _same_cache(dev[0], dev[2], ref)
        _same_cache(dev[1], dev[3], ref)
    assert float(dev[2][5, 0]) == 2.0 ** -60 and float(dev[2][1, 0]) == 1.0 and float(dev[2][2, 0]) == 2.0


def test_append_refuses_places_outside_the_cache():
    gdn = _gdn()
    kc, ks = U.make_cache(3, 2, 16, 64, _gen(2))
    x = torch.randn(4, 2, 64, generator=_gen(4)).to(BF).cuda()
    dev = [t.cuda() for t in (kc, kc.clone(), ks, ks.clone())]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(x, x, *dev, torch.tensor([48, -7, -1, 2147483647], dtype=torch.int32, device="cuda"), dev_status=st)
    assert int(st) == gdn.DEV_BAD_SLOT
    assert torch.equal(dev[0].cpu().view(torch.uint8), kc.view(torch.uint8)) and torch.equal(dev[2].cpu(), ks)
    gdn.gdn_kv8_append(x[:0], x[:0], *dev, torch.empty(0, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------- attention
def _attn_case(HK, G, D, bs, lens, news, seed, spread=0.5, nan_past=True):
    g = _gen(seed)
    N, T = len(lens), sum(news)
    need = [-(-L // bs) for L in lens]
    P, width = sum(need) + 3, max(1, max(need)) + 1
    ids = torch.randperm(P, generator=g).tolist()
    table = [[-1] * width for _ in range(N)]
    for n, m in enumerate(need):
        for p in range(m):
            table[n][p] = ids.pop()
    kc, ks = U.make_cache(P, HK, bs, D, g, spread)
    vc, vs = U.make_cache(P, HK, bs, D, g, spread)
    if nan_past:  # what a page holds past a context must not matter, NaN least of all
        for n, L in enumerate(lens):
            if L % bs:
                for c in (kc, vc):
                    c.view(torch.uint8)[table[n][L // bs], :, L % bs:] = 0x7f
    q = torch.randn(T, HK * G, D, generator=g).to(BF)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(int).tolist()
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=lens, cu=cu, max_q=max(news), HK=HK, G=G, D=D, bs=bs)


def _attn_run(c, use_cu=True, scale=None, **kw):
    gdn = _gdn()
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    st = i([0])
    lse = torch.full(c["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    q = kw.pop("q", None)
    o = gdn.gdn_kv8_attention(c["q"].cuda() if q is None else q, c["kc"].cuda(), c["vc"].cuda(), c["ks"].cuda(), c["vs"].cuda(),
                              i(c["table"]), i(c["lens"]), cu_seqlens=i(c["cu"]) if use_cu else None, max_q_len=c["max_q"],
                              scale=scale, lse=lse, dev_status=st, **kw)
    return o, lse, int(st.item())


def _attn_check(c, o, lse, scale=None):
    scale = c["D"] ** -0.5 if scale is None else scale
    ro, rl, mag = U.attention(U.f64(c["q"]), U.f64(c["kc"].float()), U.f64(c["vc"].float()), U.f64(c["ks"]), U.f64(c["vs"]),
                              c["table"], c["lens"], c["cu"], scale)
    got, gl = U.f64(o), U.f64(lse)
    assert np.array_equal(np.isnan(got), np.isnan(ro))
    fin = ~np.isnan(ro)
    tol = 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * mag + 1e-37
    bad = (np.abs(got - ro) > tol) & fin
    assert not bad.any(), f"o: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - ro) / np.maximum(mag, 1e-37)):.3e} of sum p|v|"
    empty = np.isneginf(rl)
    assert np.array_equal(empty, np.isneginf(gl)) and (got[empty] == 0).all()
    ok = np.isfinite(rl)
    assert (np.abs(gl[ok] - rl[ok]) <= 2.0 ** -17 * (1 + np.abs(rl[ok]))).all()


@pytest.mark.parametrize("HK,G,D,bs,lens,news", [
    (1, 1, 64, 16, [1], [1]), (2, 4, 128, 64, [1, 63, 64, 65, 0, 300], [1] * 6), (4, 8, 128, 16, [17, 1000, 129], [1] * 3),
    (1, 7, 64, 32, [257, 4], [1, 1]), (2, 16, 128, 128, [700, 128, 127], [1] * 3), (1, 1, 128, 64, [5000], [1]),
    (2, 8, 64, 64, [2500, 31], [1, 1]), (2, 4, 128, 64, [70, 5, 200], [4, 4, 4]), (1, 8, 128, 16, [900, 33], [4, 2]),
    (1, 5, 64, 128, [400, 3, 77], [3, 5, 0]), (2, 8, 128, 32, [1111, 64], [8, 5]), (1, 64, 128, 64, [333], [1]),
    (1, 3, 128, 64, [3000, 40], [20, 17])])
def test_attention_of_a_few_tokens(HK, G, D, bs, lens, news):
    c = _attn_case(HK, G, D, bs, lens, news, sum(lens) + D)
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)
    if all(m == 1 for m in news):
        o2, lse2, _ = _attn_run(c, use_cu=False)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3, _ = _attn_run(c)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("HK,G,D,bs,lens,news", [
    (1, 1, 128, 64, [129], [129]), (2, 4, 128, 64, [500, 64, 130], [300, 64, 1]), (1, 8, 128, 16, [257, 700], [257, 33]),
    (1, 7, 64, 32, [333, 90, 1], [150, 90, 1]), (2, 2, 64, 128, [640], [513]), (1, 4, 128, 128, [1000, 300], [100, 299]),
    (1, 16, 64, 16, [200], [77])])
def test_attention_of_many_tokens(HK, G, D, bs, lens, news):
    c = _attn_case(HK, G, D, bs, lens, news, sum(lens) + D + 1)
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)
    o3, lse3, _ = _attn_run(c)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("news", [[4, 6, 1], [150, 90, 33]])
def test_attention_rows_that_see_nothing(news):
    """Contexts shorter than the new tokens: the first tokens see nothing, their rows are 0 and -inf."""
    c = _attn_case(2, 4, 128, 16, [max(1, news[0] - 3), 0, news[2]], news, 9)
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)


@pytest.mark.parametrize("news", [[3, 4], [200, 170]])
def test_attention_nan_that_only_later_rows_see(news):
    """NaN in a key or value reaches exactly the rows, and for a value the columns, that see it."""
    lens = [news[0] + 40, news[1]]
    c = _attn_case(1, 4, 128, 64, lens, news, 21)
    at = lens[0] - 2                      # the last but one key of request 0: its first rows do not see it
    c["vc"].view(torch.uint8)[c["table"][0][at // 64], 0, at % 64, 5] = 0xff
    at = lens[0] - 1
    c["kc"].view(torch.uint8)[c["table"][0][at // 64], 0, at % 64, 9] = 0x7f
    at = 1
    c["vc"].view(torch.uint8)[c["table"][1][at // 64], 0, at % 64, 77] = 0x7f
    o, lse, st = _attn_run(c)
    got = torch.isnan(o).cpu()
    ref = torch.zeros_like(got)
    ref[news[0] - 2:news[0], :, 5] = True
    ref[news[0] - 1] = True
    ref[news[0] + 1:, :, 77] = True
    assert torch.equal(got, ref)


def test_attention_scales_of_very_different_pages():
    """Pages whose scales lie 2^80 apart, on both sides; logits in the hundreds; a tiny and a zero query."""
    c = _attn_case(2, 4, 128, 16, [200, 90], [1, 3], 33)
    e = torch.randint(-40, 40, c["vs"].shape, generator=_gen(1))
    c["vs"] = torch.ldexp(torch.ones_like(c["vs"]), e)
    c["q"][0] *= 64
    c["q"][1] = 0
    c["q"][2] = (c["q"][2].float() * 1e-30).to(BF)
    o, lse, st = _attn_run(c)
    _attn_check(c, o, lse)
    o, lse, st = _attn_run(c, scale=0.5)
    _attn_check(c, o, lse, scale=0.5)


def test_attention_query_not_finite_and_missing_pages():
    gdn = _gdn()
    c = _attn_case(1, 4, 128, 64, [130, 130], [1, 1], 41)
    c["q"][0, 1, 3] = float("inf")
    c["q"][1, 2, 3] = float("nan")
    o, lse, st = _attn_run(c)
    nan = torch.isnan(o).all(-1).cpu()
    assert nan.tolist() == [[False, True, False, False], [False, False, True, False]]
    c = _attn_case(1, 4, 128, 64, [130, 200], [1, 1], 43)
    c["table"][0][1] = -1                       # keys 64..127 are not there
    c["table"][1][0] = len(c["ks"]) + 5
    o, lse, st = _attn_run(c)
    assert st == gdn.DEV_BAD_SLOT
    _attn_check(c, o, lse)


def test_attention_bad_lengths_leave_others_alone():
    gdn = _gdn()
    c = _attn_case(1, 4, 128, 64, [130, 200], [2, 2], 44)
    o, lse, _ = _attn_run(c)
    d = dict(c)
    d["lens"] = [-1, 200]
    o2, lse2, st = _attn_run(d)
    assert st == gdn.DEV_BAD_SEQ_LEN
    # where a context is cut depends on the whole batch, so the other request is held to the 64-bit values, not to bits
    o2[:2], lse2[:2] = o[:2], lse[:2]
    _attn_check(c, o2, lse2)
    d["lens"], d["max_q"] = [130, 200], 1
    _, _, st = _attn_run(d)
    assert st == gdn.DEV_BAD_CU_SEQLENS
    d = dict(c)
    d["cu"] = [0, 3, 2]
    _, _, st = _attn_run(d)
    assert st == gdn.DEV_BAD_CU_SEQLENS


def test_attention_strided_queries_other_stream_and_graph():
    gdn = _gdn()
    c = _attn_case(2, 4, 128, 64, [300, 900, 4000], [2, 1, 3], 51)
    o, lse, _ = _attn_run(c)
    wide = torch.zeros(6, 8 * 128 + 64, dtype=BF, device="cuda")
    wide[:, :1024].copy_(c["q"].reshape(6, -1))
    o2, lse2, _ = _attn_run(c, q=wide[:, :1024].view(6, 8, 128))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    args = [c["q"].cuda(), c["kc"].cuda(), c["vc"].cuda(), c["ks"].cuda(), c["vs"].cuda(), i(c["table"]), i(c["lens"])]
    kw = dict(cu_seqlens=i(c["cu"]), max_q_len=3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o3 = gdn.gdn_kv8_attention(*args, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o3)
    out = torch.empty_like(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_kv8_attention(*args, o=out, **kw)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out)


def test_attention_in_a_cache_past_32_bit_offsets():
    """Pages whose bytes lie beyond 2^32: the same answer as from a small cache."""
    gdn = _gdn()
    c = _attn_case(2, 4, 128, 64, [500, 77], [1, 130], 61, nan_past=False)
    o, lse, _ = _attn_run(c)
    P = (1 << 32) // (2 * 64 * 128) + 64
    big = dict(c)
    shift = P - len(c["ks"])
    big["table"] = [[p + shift if p >= 0 else -1 for p in row] for row in c["table"]]
    caches = []
    for codes, sc in ((c["kc"], c["ks"]), (c["vc"], c["vs"])):
        b = torch.empty(P, 2, 64, 128, dtype=torch.float8_e4m3fn, device="cuda")
        b[shift:].view(torch.uint8).copy_(codes.view(torch.uint8))
        s = torch.ones(P, 2, device="cuda")
        s[shift:].copy_(sc)
        caches.append((b, s))
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    o2 = gdn.gdn_kv8_attention(c["q"].cuda(), caches[0][0], caches[1][0], caches[0][1], caches[1][1], i(big["table"]), i(c["lens"]),
                               cu_seqlens=i(c["cu"]), max_q_len=c["max_q"])
    assert torch.equal(o, o2)
    # and the write, to the last page
    slots = i([(P - 1) * 64 + 3])
    k = c["q"][:1, :2].cuda().contiguous()
    before = caches[0][0][P - 1].float().cpu().numpy().astype(np.float64), caches[0][1][P - 1].cpu().numpy().astype(np.float64)
    gdn.gdn_kv8_append(k, k, caches[0][0], caches[1][0], caches[0][1], caches[1][1], slots)
    ref = U.append(U.f64(k), before[0][None], before[1][None], [3])
    _same_cache(caches[0][0][P - 1:], caches[0][1][P - 1:], ref)


def test_attention_wait_that_runs_out():
    """The testing hook: every block's first wait runs out, the status says so, and the next call is right again."""
    gdn = _gdn()
    c = _attn_case(2, 4, 128, 64, [300, 90], [2, 140], 71)
    o, lse, _ = _attn_run(c)
    gdn.testing_force_wait_expiry(True)
    try:
        _, _, st = _attn_run(c)
    finally:
        gdn.testing_force_wait_expiry(False)
    assert st == gdn.DEV_WAIT_TIMEOUT
    o2, lse2, st = _attn_run(c)
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("HK,G,D,bs,lens,news", [
    (1, 8, 128, 64, [5000], [70]), (2, 4, 64, 16, [2300, 1, 2100], [65, 1, 129]), (4, 2, 128, 32, [3000, 40, 0, 2049], [33, 300, 5, 200]),
    (1, 1, 128, 128, [4100], [300]), (2, 8, 128, 64, [6000, 2500, 90], [1, 40, 70])])
def test_attention_of_many_tokens_over_long_contexts(HK, G, D, bs, lens, news):
    """Contexts long enough, and rows few enough, for tiles of rows to be cut along their keys; short requests and
    ones of a single token in the same call."""
    c = _attn_case(HK, G, D, bs, lens, news, sum(lens) + D + 2)
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)
    o3, lse3, _ = _attn_run(c)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


@pytest.mark.parametrize("HK,G,D,bs,lens,news", [
    (1, 8, 128, 64, [4], [4]), (2, 8, 128, 64, [127, 128, 129, 0, 260, 3], [4, 3, 4, 2, 0, 4]), (1, 32, 64, 16, [1, 1000], [1, 1]),
    (2, 8, 64, 32, [5000, 4], [4, 4]), (1, 6, 128, 128, [3000, 2, 640, 1281], [5, 4, 1, 5]), (4, 8, 128, 16, [7000], [4]),
    (1, 20, 128, 64, [300] * 3, [1, 1, 1])])
def test_attention_of_drafts(HK, G, D, bs, lens, news):
    """17 to 32 rows a kv head: contexts of one tile, of many, cut between blocks, empty ones."""
    c = _attn_case(HK, G, D, bs, lens, news, sum(lens) + D + 3)
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)
    o3, lse3, _ = _attn_run(c)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


def test_attention_of_many_drafts_with_nan():
    """More pairs than blocks, contexts of a tile or two, NaN past every context and one value that only the last token
    of request 7 sees."""
    rng = np.random.RandomState(9)
    news = [int(x) for x in rng.randint(0, 5, 90)]
    news[7] = 4
    lens = [int(m + x) for m, x in zip(news, rng.randint(0, 300, 90))]
    c = _attn_case(2, 8, 128, 32, lens, news, 22)
    at = lens[7] - 1
    c["vc"].view(torch.uint8)[c["table"][7][at // 32], 1, at % 32, 100] = 0x7f
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)
    assert int(torch.isnan(o).sum()) == 8


def test_attention_of_drafts_whose_weights_are_tiny():
    """One key far above 20000 others, whose weights of 2^-14 add up to more than its own."""
    c = _attn_case(1, 8, 128, 64, [20000], [4], 33, spread=0.0)
    c["kc"].view(torch.uint8).zero_()
    q = torch.zeros_like(c["q"].float())
    q[..., 0] = 1.0
    c["q"] = q.to(BF)
    page, place = c["table"][0][100 // 64], 100 % 64
    one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8)
    c["kc"].view(torch.uint8)[page, 0, place, 0] = one
    scale = 14.0 / math.log2(math.e) / float(c["ks"][page, 0])
    o, lse, st = _attn_run(c, scale=scale)
    assert st == 0
    _attn_check(c, o, lse, scale=scale)


def test_attention_of_drafts_wait_that_runs_out():
    """The testing hook on this path: a status, and the next call is right again."""
    gdn = _gdn()
    c = _attn_case(2, 8, 128, 64, [300, 900], [4, 3], 72)
    o, lse, _ = _attn_run(c)
    gdn.testing_force_wait_expiry(True)
    try:
        _, _, st = _attn_run(c)
    finally:
        gdn.testing_force_wait_expiry(False)
    assert st == gdn.DEV_WAIT_TIMEOUT
    o2, lse2, st = _attn_run(c)
    assert st == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,news", [([300, 200, 150], [100, 100, 100]), ([300, 200, 150], [100, 100, 3]),
                                       ([300, 200, 150], [100, 100, 2]), ([90, 200], [70, 1])])
def test_attention_of_prompts_whose_shortest_is_known(lens, news):
    """Tokens and bounds that do, or do not, rule out requests of few rows."""
    c = _attn_case(2, 8, 64, 32, lens, news, 61)
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)
    c["max_q"] += 40  # a looser bound: the same answer from other launches
    o2, lse2, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o2, lse2)


def test_attention_nan_in_a_cut_tile():
    """NaN values that only the last rows of a cut tile see, and a NaN key in the middle that all rows see."""
    for where in ("value", "key"):
        c = _attn_case(1, 8, 128, 64, [4000], [70], 5)
        at = 3996 if where == "value" else 1000
        c["vc" if where == "value" else "kc"].view(torch.uint8)[c["table"][0][at // 64], 0, at % 64, 5] = 0x7f
        o, lse, st = _attn_run(c)
        assert st == 0
        if where == "value":
            _attn_check(c, o, lse)
            assert torch.isnan(o[-4:, :, 5]).all() and not torch.isnan(o[:-4]).any()
        else:
            assert torch.isnan(o).all()


@pytest.mark.parametrize("N,hi,most", [(70, 900, 1), (600, 40, 1), (600, 60, 9), (40, 300, 33)])
def test_attention_of_many_requests(N, hi, most):
    """More requests than a warp, or a block, has threads; tokens from none to `most`."""
    rng = np.random.RandomState(N + most)
    news = [1] * N if most == 1 else [int(x) for x in rng.randint(0, most + 1, N)]
    lens = [int(m + x) for m, x in zip(news, rng.randint(0, hi, N))]
    c = _attn_case(1, 2 if most < 33 else 8, 64, 16, lens, news, N + hi)
    o, lse, st = _attn_run(c)
    assert st == 0
    _attn_check(c, o, lse)


def test_attention_offsets_that_go_back_are_reported():
    """cu_seqlens that count the same tokens again and again: a status, no access out of place."""
    gdn = _gdn()
    c = _attn_case(2, 8, 128, 64, [300] * 9, [20] * 9, 3)
    c["cu"], c["max_q"] = [0, 180, 0, 180, 0, 180, 0, 180, 0, 180], 180
    _, _, st = _attn_run(c)
    assert st & gdn.DEV_BAD_CU_SEQLENS


def test_rotary_embedding_of_queries_alone():
    gdn = _gdn()
    inv, _ = gdn.rope_frequencies(32, device="cuda")
    q = torch.randn(5, 2, 64, generator=_gen(4)).to(BF).cuda().requires_grad_(True)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    out, none = gdn.rotary_embedding(q, None, pos, inv)
    assert none is None
    dy = torch.randn(5, 2, 64, generator=_gen(5)).to(BF).cuda()
    (dq,) = torch.autograd.grad(out, q, dy)
    assert torch.equal(dq, gdn.gdn_rope(dy, None, pos, inv, inverse=True)[0])


def test_refusals_of_types_shapes_and_layouts():
    """Checks of the Python entries on device tensors; nothing is launched."""
    gdn = _gdn()
    x, w = torch.zeros(3, 2, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    f8 = lambda *s: torch.zeros(*s, dtype=torch.float8_e4m3fn, device="cuda")
    one = torch.ones(4, 2, device="cuda")
    cache = (f8(4, 2, 16, 64), f8(4, 2, 16, 64), one, one)
    table, lens, fr = i(0, 1, 2).view(3, 1), i(1, 1, 1), torch.ones(32, device="cuda")
    wrong = [
        (TypeError, lambda: gdn.gdn_norm_gate(x.float(), w)),
        (TypeError, lambda: gdn.gdn_norm_gate(x, w.to(BF))),
        (ValueError, lambda: gdn.gdn_norm_gate(x, w[:63])),
        (ValueError, lambda: gdn.gdn_norm_gate(x, w, z=x[:2])),
        (ValueError, lambda: gdn.gdn_norm_gate(x, w, residual=x[:, :1])),
        (ValueError, lambda: gdn.gdn_norm_gate(x.transpose(0, 1), w)),
        (ValueError, lambda: gdn.gdn_norm_gate_bwd(x, x[:2], w)),
        (TypeError, lambda: gdn.gdn_rope(x, x, torch.zeros(3, device="cuda"), fr)),
        (ValueError, lambda: gdn.gdn_rope(x, x, i(0, 1), fr)),
        (ValueError, lambda: gdn.gdn_rope(x, x[:2], i(0, 1, 2), fr)),
        (gdn.GDNError, lambda: gdn.gdn_rope(x, x, i(0, 1, 2), torch.ones(33, device="cuda"))),
        (TypeError, lambda: gdn.gdn_paged_plan(i(0).long(), i(0, 1), i(0).view(1, 1), i(0), i(1), 16, 1)),
        (ValueError, lambda: gdn.gdn_paged_plan(i(0), i(0, 1, 2), i(0).view(1, 1), i(0), i(1), 16, 1)),
        (TypeError, lambda: gdn.gdn_kv8_append(x, x, *cache, i(0, 1, 2).long())),
        (TypeError, lambda: gdn.gdn_kv8_append(x, x, cache[0].view(torch.uint8), *cache[1:], i(0, 1, 2))),
        (ValueError, lambda: gdn.gdn_kv8_append(x, x[:2], *cache, i(0, 1, 2))),
        (ValueError, lambda: gdn.gdn_kv8_append(x, x, *cache[:3], one[:3], i(0, 1, 2))),
        (TypeError, lambda: gdn.gdn_kv8_attention(x.half(), *cache, table, lens)),
        (ValueError, lambda: gdn.gdn_kv8_attention(x, *cache, table[:2], lens)),
        (ValueError, lambda: gdn.gdn_kv8_attention(x[..., :32], *cache, table, lens)),
        (gdn.GDNError, lambda: gdn.gdn_kv8_attention(x, *cache, table, lens, max_seq_len=17)),
        (gdn.GDNError, lambda: gdn.gdn_kv8_attention(x, *cache, table, lens, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]
    for n, (error, call) in enumerate(wrong):
        try:
            call()
        except error:
            continue
        except Exception as e:
            raise AssertionError(f"refusal {n}: {type(e).__name__} {e} instead of {error.__name__}")
        raise AssertionError(f"refusal {n}: accepted")


# ----------------------------------------------------- append: addresses, scales, runs
@pytest.mark.parametrize("start", [1, 2, 3, 4])
def test_append_to_a_cache_at_any_byte(start):
    """Caches that begin `start` bytes into their storage, pages whose older codes move to a larger scale."""
    gdn, g = _gdn(), _gen(80 + start)
    bs, D, H, P = 16, 64, 2, 3
    kc, ks = U.make_cache(P, H, bs, D, g)
    x = (300 * torch.randn(4, H, D, generator=g)).to(BF)
    slots = [0 * bs + 7, 0 * bs + 8, 2 * bs + 3, 1 * bs]
    held = [torch.zeros(kc.numel() + 8, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    dev = [b[start:start + kc.numel()].view(P, H, bs, D) for b in held]
    for d in dev:
        d.view(torch.uint8).copy_(kc.view(torch.uint8))
    scales = [ks.cuda(), ks.clone().cuda()]
    gdn.gdn_kv8_append(x.cuda(), x.cuda(), *dev, *scales, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    ref = U.append(U.f64(x), U.f64(kc.float()), U.f64(ks), slots)
    assert (ref[1][0] > U.f64(ks)[0]).all()  # the scale did grow
    for d, sc, b in zip(dev, scales, held):
        _same_cache(d, sc, ref)
        edge = b.view(torch.uint8)
        assert not edge[:start].any() and not edge[start + kc.numel():].any()


# ------------------------------------------------------------- plan: bad requests
def _plan_around(cached, cu, T, bad, bs, seed):
    """A batch some of whose requests are bad: the others' pages, slots and positions are those of the batch in which
    the bad ones have no new tokens, whose own slots are -1."""
    gdn, r, N = _gdn(), np.random.RandomState(seed), len(cached)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    news = [0 if n in bad else cu[n + 1] - cu[n] for n in range(N)]
    held = [0 if n in bad else c for n, c in enumerate(cached)]
    width = max(1, max(-(-(c + m) // bs) for c, m in zip(held, news)))
    ids = r.permutation(N * width + 3).tolist()
    table = [[ids.pop() if p < -(-held[n] // bs) else -1 for p in range(width)] for n in range(N)]
    start = np.concatenate([[0], np.cumsum(news)]).astype(int).tolist()
    rt, rl, rs, rp, left, missing = U.plan(held, start, table, ids, len(ids), bs, start[-1])
    assert not missing
    slots, pos = [-1] * T, [0] * T
    for n in range(N):
        for k in range(news[n]):
            slots[cu[n] + k], pos[cu[n] + k] = rs[start[n] + k], rp[start[n] + k]
    lens = [max(cached[n], 0) if n in bad else rl[n] for n in range(N)]
    t, st = i(table), i([0])
    got = gdn.gdn_paged_plan(i(cached), i(cu), t, i(ids), i([len(ids)]), bs, T, dev_status=st)
    assert int(st) & gdn.DEV_BAD_CU_SEQLENS
    for a, b in zip(got, (lens, slots, pos, [left])):
        assert a.cpu().tolist() == b
    assert t.cpu().tolist() == rt


@pytest.mark.parametrize("cached,cu,T,bad", [
    ([0, -1, 0], [0, 4, 8, 12], 12, {1}), ([0, 9, -3], [0, 5, 8, 12], 12, {2}), ([-7, 2], [0, 3, 9], 9, {0}),
    ([5, 2147483647, 3], [0, 4, 8, 12], 12, {1}),        # cached + new past int32
    ([0, 0, 0, 6], [0, 4, -7, 4, 8], 8, {1, 2}),         # a negative offset between good ones
    ([3, 1, 0, 0], [0, 4, 99, 4, 8], 8, {1, 2}),         # one past all tokens
    ([0, 5, 0], [3, 6, 8, 11], 11, {0})])                # the first offset is not 0
def test_plan_bad_requests_leave_the_others_alone(cached, cu, T, bad):
    _plan_around(cached, cu, T, bad, 4, len(cu))


@pytest.mark.parametrize("what", ["length", "offset"])
def test_plan_bad_requests_among_many(what):
    """Bad requests in the first, the middle and the last of three stretches of 1024 requests."""
    r = np.random.RandomState(5)
    N = 2500
    cached, cu = r.randint(0, 40, N).tolist(), np.concatenate([[0], np.cumsum(r.randint(0, 4, N))]).astype(int).tolist()
    T = cu[-1]
    at = [1, 500, 1023, 1024, 1700, 2499] if what == "length" else [3, 1500]
    bad = set()
    for n in at:
        if what == "length":
            cached[n] = -1 - n
            bad.add(n)
        else:
            cu[n] = -n
            bad |= {n - 1, n}
    _plan_around(cached, cu, T, bad, 16, 6)


# ---------------------------------------------------------- norm: its autograd entry
def test_norm_gate_autograd_without_a_residual_ignores_its_scale():
    """The forward without a residual does not use res_scale, and neither does its gradient."""
    gdn, g = _gdn(), _gen(12)
    x, z, dy = (torch.randn(7, 96, generator=g).to(BF) for _ in range(3))
    w = 1 + 0.1 * torch.randn(96, generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, w, z)]
    y, h = gdn.norm_gate(leaves[0], leaves[1], z=leaves[2], res_scale=0.5)
    assert h is None
    _close_bf16(y, U.norm_fwd(U.f64(x), U.f64(w), None, U.f64(z), res_scale=0.5)[0], what="y")
    dx, dw, dz = torch.autograd.grad(y, leaves, dy.cuda())
    h64 = U.f64(x)
    rx, _, rz, rw = U.norm_bwd(U.f64(dy), h64, U.f64(w), U.f64(z))
    rstd = 1 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + 1e-6)
    _close_bf16(dx, rx, 2.0 ** -18 * rstd * np.abs(U.f64(dy)).max(-1, keepdims=True) * 4, what="dx")
    _close_bf16(dz, rz, 2.0 ** -18 * np.abs(U.f64(dy) * h64 * rstd), what="dz")
    mags = np.abs(U.f64(dy) * h64 * rstd * U.act(U.f64(z), "silu")[0]).sum(0)
    assert (np.abs(U.f64(dw) - rw) <= 2.0 ** -19 * mags + 1e-30).all()


# ------------------------------------------------------------- second derivatives
@pytest.mark.parametrize("entry", ["norm_gate", "rotary_embedding", "chunk_gated_delta_rule"])
def test_second_derivatives_are_refused(entry):
    """The gradients come from kernels that have none of their own: with another differentiable path beside them the
    second derivative would miss a term, so it raises.  First derivatives with create_graph stay what they are."""
    gdn, g = _gdn(), _gen(13)
    x = torch.randn(1, 8, 2, 64, generator=g).to(BF).cuda().requires_grad_()
    if entry == "norm_gate":
        w = torch.ones(64, device="cuda")
        call = lambda: gdn.norm_gate(x, w)[0]
    elif entry == "rotary_embedding":
        inv, _ = gdn.rope_frequencies(64, device="cuda")
        pos = torch.arange(8, dtype=torch.int32, device="cuda")
        call = lambda: gdn.rotary_embedding(x[0], None, pos, inv)[0]
    else:
        gates = torch.rand(1, 8, 2, generator=g).cuda()
        k = torch.randn(1, 8, 2, 64, generator=g).to(BF).cuda()
        call = lambda: gdn.chunk_gated_delta_rule(x, k, k, -gates, gates, output_final_state=False)[0]
    (plain,) = torch.autograd.grad(call().float().square().sum(), x)
    (dx,) = torch.autograd.grad(call().float().square().sum(), x, create_graph=True)
    assert torch.equal(dx, plain)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dx.float().square().sum() + x.float().square().sum()).backward()


@pytest.mark.parametrize("D,bs", [(64, 16), (10, 5)])
def test_append_to_pages_whose_scale_is_no_power_of_two(D, bs):
    """Pages from elsewhere: their older tokens keep their values, rounded once to the page's new scale, whether that
    scale comes from the old one (small new tokens) or from the new tokens (large ones)."""
    gdn, g = _gdn(), _gen(90 + D)
    # few significant bits, so that a code times such a scale is exact in fp32
    before = torch.tensor([0.75, 1.25, 1.9375 * 2.0 ** -30, 1.5 * 2.0 ** -70, 2.0 ** -100, 3.0, 2.0 ** 122, 0.0, 0.25])
    P = len(before)
    codes = (60 * torch.randn(P, 1, bs, D, generator=g)).to(torch.float8_e4m3fn)
    ks = before[:, None].clone()
    x = torch.randn(2 * P, 1, D, generator=g)
    x[1::2] *= 3000.0
    for n, rows in enumerate((x[::2].to(BF), x[1::2].to(BF))):
        off = 2 + n
        slots = [p * bs + off for p in range(P)]
        dev = [codes.cuda(), codes.clone().cuda(), ks.cuda(), ks.clone().cuda()]
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_kv8_append(rows.cuda(), rows.cuda(), *dev, torch.tensor(slots, dtype=torch.int32, device="cuda"), dev_status=st)
        assert int(st) == 0
        rc, rs = U.f64(codes.float()), U.f64(ks)
        for p in range(P):
            s = float(before[p])
            m, e = math.frexp(s)
            over = U.EXP_MIN if s == 0 else max(U.EXP_MIN, e - 1 if m == 0.5 else e)
            e = max(over, U.least_exponent(float(rows[p].float().abs().max())))
            rc[p, 0, :off] = U.to_e4m3(rc[p, 0, :off] * s * 2.0 ** -e)
            rc[p, 0, off] = U.to_e4m3(U.f64(rows[p, 0]) * 2.0 ** -e)
            rs[p, 0] = 2.0 ** e
        for d, sc in ((dev[0], dev[2]), (dev[1], dev[3])):
            _same_cache(d, sc, (rc, rs))


@pytest.mark.parametrize("kind", ["silu", "sigmoid"])
@pytest.mark.parametrize("res", [False, True])
def test_norm_gate_and_gradients_of_an_empty_batch(kind, res):
    gdn = _gdn()
    e, w = torch.empty(0, 2, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (e, w, e)] + ([e.clone().requires_grad_()] if res else [])
    y, h = gdn.norm_gate(leaves[0], leaves[1], z=leaves[2], residual=leaves[3] if res else None, activation=kind)
    assert y.shape == e.shape and (h.shape == e.shape if res else h is None)
    grads = torch.autograd.grad([y, h] if res else y, leaves, [e, e] if res else e)
    assert [g.shape for g in grads] == [t.shape for t in leaves] and (grads[1] == 0).all()


def test_plan_reports_tokens_on_a_page_that_an_earlier_step_did_not_get():
    """A step that runs out of pages says so, and so does the next one, whose tokens fall on the missing page."""
    gdn = _gdn()
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    t, st = i([[-1, -1], [4, -1]]), i([0])
    cu = i([0, 3, 4])
    lens, slots, pos, left = gdn.gdn_paged_plan(i([0, 1]), cu, t, i([9]), i([0]), 16, 4, dev_status=st)
    assert int(st) == gdn.DEV_NO_PAGE and slots.tolist() == [-1, -1, -1, 4 * 16 + 1]
    st.zero_()
    lens, slots, pos, left = gdn.gdn_paged_plan(lens, cu, t, i([9]), i([1]), 16, 4, dev_status=st)
    assert int(st) == gdn.DEV_NO_PAGE and slots.tolist() == [-1, -1, -1, 4 * 16 + 2] and pos.tolist() == [3, 4, 5, 2]
    assert t.tolist() == [[-1, -1], [4, -1]] and left.tolist() == [1]


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("places", [[3, -1, 4], [3, 3], [4, 3], [15, 0], [3] + 31 * [-1] + [4], [3, 5], [3, -1, 4, 5, -1, 6]])
def test_append_leaves_out_a_second_run_of_a_page(places, many):
    """A rejected token in the middle of a draft, a hole, a repeated place: the first run is written, the rest is left out
    and reported; other pages get theirs.  `many`: enough tokens for blocks of four warps."""
    gdn, g = _gdn(), _gen(len(places))
    bs, D, H, lead = 16, 64, 8 if many else 2, 900 if many else 2
    P = -(-lead // bs) + 3
    slots = list(range(lead)) + [(P - 2) * bs + p if p >= 0 else -1 for p in places] + [(P - 1) * bs + 7, (P - 1) * bs + 8]
    first = 1
    while first < len(places) and places[first] == places[0] + first and places[first]:
        first += 1
    kept = list(slots)
    kept[lead + first:lead + len(places)] = [-1] * (len(places) - first)
    kc, ks = U.make_cache(P, H, bs, D, g)
    x = (3 * torch.randn(len(slots), H, D, generator=g)).to(BF)
    dev = [t.cuda() for t in (kc, kc.clone(), ks, ks.clone())]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(x.cuda(), x.cuda(), *dev, torch.tensor(slots, dtype=torch.int32, device="cuda"), dev_status=st)
    assert int(st) == gdn.DEV_BAD_SLOT
    ref = U.append(U.f64(x), U.f64(kc.float()), U.f64(ks), kept)
    _same_cache(dev[0], dev[2], ref)
    _same_cache(dev[1], dev[3], ref)


# --------------------------------------------------------- attention: far weights
@pytest.mark.parametrize("G,D,N,news,ctx", [(8, 128, 700, 1, 3000), (16, 64, 700, 1, 3000), (8, 128, 1, 70, 3000), (8, 64, 1, 70, 3000),
                                            (8, 128, 160, 4, 3000)])
@pytest.mark.parametrize("bits", [20.0, 25.1, 28.0])
def test_attention_of_a_key_far_above_all_others(G, D, N, news, ctx, bits):
    """A key at the context's beginning whose weight is 2^bits of the others' and whose value is 0: the result is the
    others' mean times their mass.  700 requests (of the same pages), so that a team has many stages of one context.
    Beside the bound of the other tests a weight may be off by 2^-36 of the largest (17 to 32 rows a request: 2^-29)."""
    c = _attn_case(1, G, D, 64, [ctx], [news], 5, spread=0.0)
    c["kc"].view(torch.uint8).zero_()
    c["vc"].view(torch.uint8).bitwise_and_(0x7f)  # values of one sign, which do not cancel
    q = torch.zeros_like(c["q"].float())
    q[..., 0] = 1.0
    c["q"] = q.to(BF)
    page = c["table"][0][0]
    c["kc"].view(torch.uint8)[page, 0, 20, 0] = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8)
    c["vc"].view(torch.uint8)[page, 0, 20] = 0
    scale = bits / math.log2(math.e) / float(c["ks"][page, 0])
    args = [U.f64(c[k].float() if k in ("kc", "vc") else c[k]) for k in ("q", "kc", "vc", "ks", "vs")]
    ref, rl, mag = U.attention(*args, c["table"], c["lens"], c["cu"], scale)
    v = np.concatenate([args[2][p, 0] * args[4][p, 0] for p in c["table"][0][:-(-ctx // 64)]])[:ctx]
    c["table"], c["lens"], c["q"] = c["table"] * N, c["lens"] * N, c["q"].repeat(N, 1, 1)
    c["cu"] = [news * n for n in range(N + 1)]
    o, lse, st = _attn_run(c, scale=scale)
    assert st == 0
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + 2.0 ** (-29 if 16 < news * G <= 32 else -36) * np.abs(v).sum(0)
    off = np.abs(U.f64(o).reshape(N, *ref.shape) - ref)
    assert (off <= tol).all(), f"worst {(off / np.abs(ref)).max():.3f} of the value"
    assert (np.abs(U.f64(lse).reshape(N, *rl.shape) - rl) <= 2.0 ** -17 * (1 + np.abs(rl))).all()


@pytest.mark.parametrize("news", [1, 2, 4, 70])
@pytest.mark.parametrize("top", [1.5 * 2 ** 20, 1.1 * 2 ** 26, 1.6 * 2 ** 26, 1.3 * 2 ** 27, 1.9 * 2 ** 27, 1.2 * 2 ** 28])
def test_attention_of_very_large_logits(news, top):
    """Exponents (base 2) whose fp32 steps are as wide as f16 is high: one key has all the weight, nothing overflows."""
    c = _attn_case(1, 8, 128, 64, [700], [news], 6, spread=0.0)
    c["kc"].view(torch.uint8).zero_()
    q = torch.zeros_like(c["q"].float())
    q[..., 0] = 1.0
    c["q"] = q.to(BF)
    for key, val in ((5, 0.75), (300, 1.0), (620, 0.875)):
        c["kc"].view(torch.uint8)[c["table"][0][key // 64], 0, key % 64, 0] = torch.tensor(val).to(torch.float8_e4m3fn).view(torch.uint8)
    c["ks"][:] = 1.0
    scale = float(np.float32(top / math.log2(math.e)))
    o, lse, st = _attn_run(c, scale=scale)
    assert st == 0
    _attn_check(c, o, lse, scale=scale)


def test_outputs_that_do_not_fit_raise_the_out_of_memory_error():
    """The error that a program catches to free its caches and try again (the process' share of the memory is made
    small for the call; nothing is allocated)."""
    gdn = _gdn()
    T = 1 << 16
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # before q too, which would take a part of a larger block and leave the rest free
    inv, _ = gdn.rope_frequencies(64, device="cuda")
    q, pos = torch.zeros(T, 8, 64, dtype=BF, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() / torch.cuda.get_device_properties(0).total_memory)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            gdn.gdn_rope(q, None, pos, inv)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(gdn.gdn_rope(q, None, pos, inv)[0], q)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_calls_go_to_the_tensors_device():
    """Tensors of a device that is not the current one: the call runs there."""
    gdn = _gdn()
    x, w = torch.randn(9, 128, generator=_gen(3)).to(BF), torch.ones(128)
    here = gdn.gdn_norm_gate(x.to("cuda:0"), w.to("cuda:0"))[0]
    assert torch.cuda.current_device() == 0
    there = gdn.gdn_norm_gate(x.to("cuda:1"), w.to("cuda:1"))[0]
    assert torch.cuda.current_device() == 0 and there.device.index == 1 and torch.equal(here.cpu(), there.cpu())


@pytest.mark.parametrize("lead,heads", [((3, 5), (4,)), ((3, 5), ()), ((2, 3, 4), (2,)), ((1, 7), (1,)), ((6,), (2, 3))])
def test_norm_gate_of_a_packed_projection_with_a_batch(lead, heads):
    """A gate that is a slice of a projection [.., tokens, width], whatever dimensions stand before the tokens."""
    gdn, g = _gdn(), _gen(41)
    D, H = 64, math.prod(heads)
    wide = torch.randn(*lead, 2 * H * D + 8, generator=g).to(BF).cuda()
    z = wide[..., H * D:2 * H * D].unflatten(-1, (*heads, D))
    assert not z.is_contiguous() or math.prod(lead) == 1
    x, dy = (torch.randn(*lead, *heads, D, generator=g).to(BF).cuda() for _ in range(2))
    w = 1 + torch.rand(D, generator=g).cuda()
    a, b = gdn.gdn_norm_gate(x, w, z=z)[0], gdn.gdn_norm_gate(x, w, z=z.contiguous())[0]
    assert torch.equal(a, b)
    a, b = gdn.gdn_norm_gate_bwd(dy, x, w, z=z), gdn.gdn_norm_gate_bwd(dy, x, w, z=z.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(a, b) if p is not None)


def test_norm_gate_refuses_gates_whose_tokens_are_not_evenly_apart():
    gdn = _gdn()
    w, x = torch.ones(64, device="cuda"), torch.zeros(3, 5, 2, 64, dtype=BF, device="cuda")
    wide = torch.zeros(3, 7, 4, 128, dtype=BF, device="cuda")
    for z in (wide[:, :5, :2, :64], wide[:, :5, :2, ::2]):
        with pytest.raises(ValueError, match="longer stride"):
            gdn.gdn_norm_gate(x, w, z=z)



# --------------------------------------- append: blocks of four warps, one for a page's length of tokens
def _many_runs(bs, T, r):
    """Slots of ragged requests on pages of their own, skipped tokens between some, T tokens or a few more; and pages."""
    slots, pages = [], 0
    while len(slots) < T:
        if r.rand() < 0.2:
            slots += [-1] * int(r.randint(1, 6))
        off = int(r.randint(0, bs))
        m = int(r.choice([1, 2, 3, int(r.randint(1, bs + 1)), int(r.randint(1, 4 * bs))]))
        slots += range(pages * bs + off, pages * bs + off + m)
        pages += -(-(off + m) // bs)
    names = r.permutation(pages)
    return [-1 if s < 0 else int(names[s // bs]) * bs + s % bs for s in slots], pages


@pytest.mark.parametrize("HK,D,bs", [(8, 128, 16), (8, 64, 16), (8, 128, 32), (8, 64, 64), (4, 128, 64), (8, 128, 48), (8, 64, 128),
                                     (8, 128, 128), (4, 512, 8), (16, 32, 128), (16, 16, 64), (4, 256, 16)])
def test_append_of_many_tokens(HK, D, bs):
    """Enough tokens for the kernel that long prompts take, with each number of values that its threads hold: runs that
    begin anywhere in a page, cross the blocks' stretches, or are short; older codes that move; values that are not finite."""
    gdn, g, r = _gdn(), _gen(HK + D + bs), np.random.RandomState(HK + D + bs)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    slots, P = _many_runs(bs, bs * -(-4 * sms // (2 * HK)) + 5, r)
    T = len(slots)
    assert -(-T // bs) * 2 * HK >= 4 * sms
    kc, ks = U.make_cache(P, HK, bs, D, g)
    vc, vs = U.make_cache(P, HK, bs, D, g)
    wide = torch.randn(T, 2 * HK * D, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))
    for bad in (math.inf, -math.inf, math.nan):
        wide.view(-1)[torch.randint(0, wide.numel(), (20,), generator=g)] = bad
    wide = wide.to(BF)
    k, v = (wide[:, i * HK * D:(i + 1) * HK * D].view(T, HK, D) for i in range(2))
    wd = wide.cuda()
    kd, vd = (wd[:, i * HK * D:(i + 1) * HK * D].view(T, HK, D) for i in range(2))
    dev = [t.cuda() for t in (kc, vc, ks, vs)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv8_append(kd, vd, *dev, torch.tensor(slots, dtype=torch.int32, device="cuda"), dev_status=st)
    assert int(st) == 0
    _same_cache(dev[0], dev[2], U.append(U.f64(k), U.f64(kc.float()), U.f64(ks), slots))
    _same_cache(dev[1], dev[3], U.append(U.f64(v), U.f64(vc.float()), U.f64(vs), slots))


# ------------------------------------------- norms: more rows than the blocks take in one turn
def _act64(z, kind):
    s = 1.0 / (1.0 + (-z).exp())
    return (z * s, s * (1.0 + z * (1.0 - s))) if kind == "silu" else (s, s * (1.0 - s))


@pytest.mark.parametrize("rows,D", [(100003, 64), (50021, 128), (30011, 256), (25013, 512), (25013, 1024), (3001, 2048), (3001, 4096),
                                    (1517, 8192), (1517, 16384), (3001, 130), (2999, 1001)])
@pytest.mark.parametrize("kind,res", [(None, False), ("silu", True), ("sigmoid", False)])
def test_norm_gate_and_gradients_of_many_rows(rows, D, kind, res):
    """Every kernel in several turns, the last one not full: a turn is 38912 rows of 64 forward, and down to 608 rows of
    16384 (backward 19456, and 152).  The formulas in 64 bits by torch.  Tolerances as above; the weight's gradient is
    a chain of at most 128 additions (turns, row groups of a block, blocks): 2^-17 of the magnitudes."""
    gdn = _gdn()
    gen = torch.Generator(device="cuda").manual_seed(rows + D)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy, s = (2 * rnd(rows, D)).to(BF), rnd(rows, D).to(BF), 0.5 if res else 1.0
    w = 1 + 0.1 * rnd(D)
    z = rnd(rows, D).to(BF) if kind else None
    r, dh = (rnd(rows, D).to(BF), rnd(rows, D).to(BF)) if res else (None, None)

    def close(got, ref, extra, what):
        off = (got.double() - ref).abs() - (2.0 ** -8 * ref.abs() + extra + 1e-37)
        assert float(off.max()) <= 0, f"{what}: {int((off > 0).sum())} of {off.numel()}"

    y, h = gdn.gdn_norm_gate(x, w, residual=r, z=z, activation=kind, res_scale=s)
    h64 = x.double() if r is None else r.double() + s * x.double()
    f, d = (1.0, None) if kind is None else _act64(z.double(), kind)
    close(y, h64 / (h64.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double() * f, 0.0, "y")
    if res:
        close(h, h64, 2.0 ** -18 * float(h64.abs().max()), "h")
    hb = x if h is None else h
    grads = gdn.gdn_norm_gate_bwd(dy, hb, w, z=z, dh=dh, activation=kind, res_scale=s)
    again = gdn.gdn_norm_gate_bwd(dy, hb, w, z=z, dh=dh, activation=kind, res_scale=s)
    assert all(torch.equal(a, b) for a, b in zip(grads, again) if a is not None)
    dx, dres, dz, dw = grads
    h64 = hb.double()
    rstd = 1.0 / (h64.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    n = h64 * rstd
    u = dy.double() * f
    p = u * w.double()
    dH = rstd * (p - n * (p * n).mean(-1, keepdim=True)) + (0.0 if dh is None else dh.double())
    terms = 2.0 ** -18 * (rstd * dy.double().abs().amax(-1, keepdim=True) * 4 + (2.0 if res else 0.0))
    close(dx, s * dH, terms, "dx")
    if res:
        close(dres, dH, terms, "dresidual")
    if kind:
        close(dz, dy.double() * n * w.double() * d, 2.0 ** -18 * (dy.double() * n).abs(), "dz")
    assert ((dw.double() - (u * n).sum(0)).abs() <= 2.0 ** -17 * (u * n).abs().sum(0)).all()


# ---------------------------------- attention: more tiles of rows than SMs, so whole ones come before those cut
def _attn64(c, scale):
    """o, lse and sum_j p_ij |v_j| in 64 bits by torch, one product a (request, kv head)."""
    HK, G, D, bs = c["HK"], c["G"], c["D"], c["bs"]
    q, ks, vs = (c[k].cuda().double() for k in ("q", "ks", "vs"))
    o, mag, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for n, L in enumerate(c["lens"]):
        t0, t1 = c["cu"][n], c["cu"][n + 1]
        m = t1 - t0
        pages = torch.tensor(c["table"][n][:-(-L // bs)], device="cuda")
        seen = torch.arange(L, device="cuda") <= torch.arange(L - m, L, device="cuda").repeat_interleave(G)[:, None]
        for h in range(HK):
            K, V = ((codes.cuda().float().double()[pages, h] * s[pages, h][:, None, None]).reshape(-1, D)[:L]
                    for codes, s in ((c["kc"], ks), (c["vc"], vs)))
            s = (q[t0:t1, h * G:(h + 1) * G].reshape(m * G, D) @ K.T * scale).masked_fill(~seen, -math.inf)
            lse[t0:t1, h * G:(h + 1) * G] = s.logsumexp(-1).view(m, G)
            p = s.sub_(s.logsumexp(-1, keepdim=True)).exp_()
            o[t0:t1, h * G:(h + 1) * G] = (p @ V).view(m, G, D)
            mag[t0:t1, h * G:(h + 1) * G] = (p @ V.abs()).view(m, G, D)
    return o, lse, mag


@pytest.mark.parametrize("HK,G,D,bs,lens,news,most", [
    (2, 8, 128, 64, [2500, 5000], [2450, 300], 152),               # 174 tiles: 152 whole, 22 in 5 pieces
    (4, 4, 64, 16, [3000, 2100, 4200], [3000, 2000, 200], 304),     # 332: two turns whole, 28 in 4 pieces
    (1, 8, 64, 128, [4864], [4864], 152),                           # one tile an SM, none left
    (1, 8, 128, 32, [8064, 3], [8064, 3], 152)])                    # 253: 101 left, too many to cut
def test_attention_of_more_tiles_of_rows_than_sms(HK, G, D, bs, lens, news, most):
    c = _attn_case(HK, G, D, bs, lens, news, sum(lens) + D, nan_past=False)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert HK * sum(-(-m * G // 256) for m in news) >= most
    o, lse, st = _attn_run(c)
    assert st == 0
    ro, rl, mag = _attn64(c, D ** -0.5)
    off = (o.double() - ro).abs() - (2.0 ** -8 * ro.abs() + 2.0 ** -10 * mag + 1e-37)
    assert float(off.max()) <= 0, f"{int((off > 0).sum())} of {off.numel()}"
    assert ((lse.double() - rl).abs() <= 2.0 ** -17 * (1 + rl.abs())).all()
    again, lse2, _ = _attn_run(c)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("news", [1, 2, 4, 70])
def test_attention_scales_at_the_ends_of_their_range(news):
    """Values in pages of scale 2^-90, and of 2^100, alone: neither the sum of the weights nor the result overflows."""
    for e in (-90, 100):
        c = _attn_case(1, 8, 128, 64, [3000], [news], 7)
        c["vs"] = torch.full_like(c["vs"], 2.0 ** e)
        o, lse, st = _attn_run(c)
        assert st == 0 and torch.isfinite(o).all()
        _attn_check(c, o, lse)

