"""The hybrid stack's training path on packed sequences: outputs and gradients against the same stack in plain 64-bit torch
operations.

Bounds, as the length of the difference over the length of the value.  A rounding to bf16 is off by 2^-8 at most and about
2^-9.5 as a root mean square; some twenty follow one another on the way through three layers and back, and they add as
squares: 20^(1/2) 2^-9.5 = 0.6 %, the norms' and gates' slopes some more: 4 %.  An 8-bit code is off by 2^-4 at most, 2.6 %
as a root mean square; a weight's gradient takes one such input, a stream's those of the norms after it, seven in all:
12 %."""
import math

import pytest
import torch
import torch.nn.functional as nn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_chunked_chunk_gb300 import build
    build.build()


def _rms(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def _rope(x, inv_freq):
    rot = 2 * inv_freq.numel()
    t = torch.arange(x.shape[0], device=x.device, dtype=x.dtype)[:, None, None] * inv_freq
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos(), x[..., rot:]), -1)


def _plain(stack, params, x, lens):
    cfg, it = stack.cfg, iter(params)
    last = next(it)
    h, y = x, None
    for layer in stack.layers:
        norm, w_in, w_out = next(it), next(it), next(it)
        h = h if y is None else h + y
        u = _rms(h, norm) @ w_in.T
        outs = []
        if layer.kind == "a":
            for part in u.split(lens):
                m = part.shape[0]
                q, k, v = part.view(m, -1, cfg.D).split([cfg.HQ, cfg.HK, cfg.HK], dim=1)
                q, k = (_rope(t, stack.inv_freq.double()) for t in (q, k))
                k, v = (t.repeat_interleave(cfg.HQ // cfg.HK, dim=1) for t in (k, v))
                s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(cfg.D)
                s = s.masked_fill(torch.ones(m, m, dtype=torch.bool, device=x.device).triu(1), -math.inf)
                outs.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(m, -1))
        else:
            out_norm = next(it)
            for part in u.split(lens):
                q, k, v, z, a, b = part.split([cfg.H * cfg.K, cfg.H * cfg.K, cfg.HV * cfg.K, cfg.HV * cfg.K, cfg.HV, cfg.HV], dim=1)
                q, k, v, z = (t.unflatten(1, (-1, cfg.K)) for t in (q, k, v, z))
                q, k = (t * torch.rsqrt(t.square().sum(-1, keepdim=True) + 1e-6) for t in (q, k))
                q, k = (t.repeat_interleave(cfg.HV // cfg.H, dim=1) for t in (q, k))
                decay = torch.exp(-layer.A_log.double().exp() * nn.softplus(a + layer.dt_bias.double()))
                beta, state, rows = b.sigmoid(), x.new_zeros(cfg.HV, cfg.K, cfg.K), []
                for t in range(part.shape[0]):
                    state = state * decay[t, :, None, None]
                    change = beta[t, :, None] * (v[t] - torch.einsum("hkv,hk->hv", state, k[t]))
                    state = state + k[t, :, :, None] * change[:, None]
                    rows.append(torch.einsum("hkv,hk->hv", state, q[t]) / math.sqrt(cfg.K))
                outs.append((_rms(torch.stack(rows), out_norm) * z * z.sigmoid()).reshape(part.shape[0], -1))
        y = torch.cat(outs) @ w_out.T
    return _rms(h + y, last)


@pytest.mark.parametrize("save8,bound", [(False, 0.04), (True, 0.12)])
def test_gradients_of_packed_sequences(save8, bound):
    from gated_deltanet_chunked_chunk_gb300.hybrid import HybridStack
    lens = [40, 1, 23]
    gen = torch.Generator().manual_seed(11)
    x, up = (torch.randn(sum(lens), 512, generator=gen).to("cuda", BF) for _ in range(2))
    stack = HybridStack(requests=1, seed=4)
    params = [p.requires_grad_(True) for p in stack.parameters()]
    out = stack.forward(x, lens, save8)
    grads = torch.autograd.grad(out, params, up)
    exact = [p.detach().double().requires_grad_(True) for p in params]
    want = _plain(stack, exact, x.double(), lens)
    ref = torch.autograd.grad(want, exact, up.double())

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    assert off(out.detach(), want.detach()) < 0.04  # the forward is the same either way
    for i, (g, r) in enumerate(zip(grads, ref)):
        assert g.shape == r.shape and off(g, r) < bound, (i, tuple(g.shape), off(g, r))


def test_packed_sequences_are_those_alone():
    """A sequence's outputs do not depend on what it is packed with, but for the last bits of sums whose order the batch's
    shape sets (a matrix product's): 1 %."""
    from gated_deltanet_chunked_chunk_gb300.hybrid import HybridStack
    lens = [70, 130, 1]
    gen = torch.Generator().manual_seed(12)
    x = torch.randn(sum(lens), 512, generator=gen).to("cuda", BF)
    stack = HybridStack(requests=1, seed=5)
    with torch.no_grad():
        packed = stack.forward(x, lens).split(lens)
        for a, b in zip(packed, x.split(lens)):
            alone = stack.forward(b)
            assert float((a.float() - alone.float()).norm() / alone.float().norm()) < 0.01


def _one_sequence(stack, x):
    """The stack on one sequence with fp32 attention from elementary operations, as it is without lengths."""
    from gated_deltanet_chunked_chunk_gb300 import norm_gate, rotary_embedding
    cfg, T = stack.cfg, x.shape[0]
    positions = torch.arange(T, dtype=torch.int32, device=x.device)
    h, y = x, None
    for layer in stack.layers:
        n, h = (norm_gate(h, layer.norm)[0], h) if y is None else norm_gate(y, layer.norm, residual=h)
        q, k, v = (n @ layer.w_in.T).view(T, -1, cfg.D).split([cfg.HQ, cfg.HK, cfg.HK], dim=1)
        q, k = rotary_embedding(q, k, positions, stack.inv_freq, attention_factor=stack.rope_factor)
        k, v = (t.repeat_interleave(cfg.HQ // cfg.HK, dim=1).transpose(0, 1).float() for t in (k, v))
        s = q.transpose(0, 1).float() @ k.transpose(1, 2) / math.sqrt(cfg.D)
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=x.device).triu(1), -math.inf)
        y = (s.softmax(-1) @ v).transpose(0, 1).to(BF).reshape(T, -1) @ layer.w_out.T
    return norm_gate(y, stack.norm, residual=h)[0]


@pytest.mark.parametrize("D,rotary", [(128, 64), (64, 64), (32, 32), (96, 64), (256, 64)])
def test_one_sequence_has_fp32_attention(D, rotary):
    """Without lengths the attention's logits, weights and their gradients stay in fp32, for heads of any size: the very
    results of the elementary operations."""
    from gated_deltanet_chunked_chunk_gb300.hybrid import Config, HybridStack
    gen = torch.Generator().manual_seed(13)
    x, up = (torch.randn(150, 512, generator=gen).to("cuda", BF) for _ in range(2))
    stack = HybridStack(Config(layers="aa", D=D, rotary=rotary), requests=1, seed=6)
    params = [p.requires_grad_(True) for p in stack.parameters()]
    got, want = (f(x) for f in (stack.forward, lambda t: _one_sequence(stack, t)))
    assert torch.equal(got, want)
    for a, b in zip(torch.autograd.grad(got, params, up), torch.autograd.grad(want, params, up)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("save8", [False, True])
def test_packed_sequences_with_other_heads(save8):
    """Heads that the kernels do not take: each sequence as it is alone, but for the batch's shape in matrix products (1 %)."""
    from gated_deltanet_chunked_chunk_gb300.hybrid import Config, HybridStack
    lens = [70, 1, 79]
    gen = torch.Generator().manual_seed(14)
    x = torch.randn(sum(lens), 512, generator=gen).to("cuda", BF)
    stack = HybridStack(Config(layers="ga", D=32, rotary=32), requests=1, seed=6)
    with torch.no_grad():
        for a, b in zip(stack.forward(x, lens, save8).split(lens), x.split(lens)):
            alone = stack.forward(b)
            assert float((a.float() - alone.float()).norm() / alone.float().norm()) < 0.01


def test_forward_of_one_sequence_is_captured():
    """Nothing of it comes from the host."""
    from gated_deltanet_chunked_chunk_gb300.hybrid import HybridStack
    gen = torch.Generator().manual_seed(15)
    x = torch.randn(130, 512, generator=gen).to("cuda", BF)
    stack = HybridStack(requests=1, seed=7)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.no_grad():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = stack.forward(x)
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            out = stack.forward(x)
        out.zero_()
        graph.replay()
    assert torch.equal(out, want)


def test_lengths_that_are_not_those_of_the_tokens():
    from gated_deltanet_chunked_chunk_gb300.hybrid import Config, HybridStack
    stack = HybridStack(Config(layers="g"), requests=1, seed=8)
    x = torch.zeros(10, 512, dtype=BF, device="cuda")
    for lens in ([], [4], [4, 7], [12, -2], [11, 0]):
        with pytest.raises(ValueError, match="lens"):
            stack.forward(x, lens)
    with torch.no_grad():
        assert torch.equal(stack.forward(x, (4, 0, 6)), stack.forward(x, [4, 0, 6]))


def _kept(stack, T, save8):
    """Bytes of all storages that the graph of a forward keeps."""
    held = {}

    def pack(t):
        held[t.untyped_storage().data_ptr()] = t.untyped_storage().nbytes()
        return t

    for p in stack.parameters():
        p.requires_grad_(True)
    x = torch.randn(T, 512, generator=torch.Generator().manual_seed(16)).to("cuda", BF)
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        out = stack.forward(x, [T], save8)
    total = sum(held.values())
    del out
    return total


@pytest.mark.parametrize("layers,bf16,save8", [
    # bf16: the stream twice, the input, the projection, rotated q and k, o and lse; save8: three codes, q, k, v, o and lse
    ("a", 2 * 1024 + 1024 + 12 * 256 + 2560 + 2048 + 32, 3 * 528 + 12 * 256 + 2048 + 32),
    # bf16: the stream twice, the input, the projection (for z), q, k, v, the recurrence's output, the normed one; save8:
    # three codes of the stream and the input, q, k, v, three codes of 8 heads of 128 (o, z and the projection's input);
    # both: gates in fp32
    ("g", 2 * 1024 + 1024 + 6176 + 4096 + 2048 + 2048, 3 * 528 + 4096 + 3 * 1056),
])
def test_bytes_that_a_step_keeps(layers, bf16, save8):
    """What save8 is for: bytes a token that the forward keeps for the gradients (positions, and the few numbers of the
    gates' formulas, 8 of 4 bytes each a head, come on top)."""
    from gated_deltanet_chunked_chunk_gb300.hybrid import Config, HybridStack
    stack = HybridStack(Config(layers=layers), requests=1, seed=9)
    few = 8 + (0 if layers == "a" else 8 * 4 * 8)
    for on, want in ((False, bf16), (True, save8)):
        got = (_kept(stack, 768, on) - _kept(stack, 256, on)) / 512
        assert want <= got <= want + few, (on, got, want)
