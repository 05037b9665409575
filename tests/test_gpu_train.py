"""A training step's attention on the GPU against plain 64-bit implementations (tests/train_util.py).

Tolerances, from the roundings.  A bf16 result is off by half a step, 2^-8 of its value.  The softmax weights, and the
gradients of the logits, enter the products in bf16: 2^-8 of each term, so 2^-8 of the sum of the terms' magnitudes.
What stays in fp32: a logit is a sum of D products, off by some D 2^-24 = 2^-17 of the sum of their magnitudes M (the
tensor cores may cut instead of round, twice that), and that is the relative error of its weight, beside 2^-21 of the
hardware's exponential; delta and dP likewise.  2^-15 (1 + M) of the terms' magnitudes covers their sum.  The gradient
takes o in bf16, as the forward gave it: delta is off by 2^-8 sum |do o|, which is a term like the rounded ones."""
import math

import pytest
import torch

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
