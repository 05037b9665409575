"""A small hybrid stack, to show how the operators are used together: gated-delta-rule layers and attention layers in
turn, each behind a norm with a residual, random weights.

    python -m gated_deltanet_chunked_chunk_gb300.hybrid

serves a few ragged prompts (prefill, then single tokens) with a state pool for the recurrence and a paged 8-bit cache
for the attention, and runs training steps: on one sequence, and on packed ones with the inputs that the gradients need
kept in bf16 and in 8 bits.  Projections are plain matrix products."""
from __future__ import annotations

import argparse
import dataclasses
import math
from typing import List, Optional

import torch

from . import (attention, chunk_gated_delta_rule, gdn_causal_conv1d_fwd, gdn_chunk_fwd_gated, gdn_conv_decode_pack, gdn_kv8_append,
               gdn_kv8_attention, gdn_norm_gate, gdn_paged_plan, gdn_recurrent_decode, gdn_rope, linear8,
               norm_gate, rope_frequencies, rotary_embedding)

BF = torch.bfloat16


@dataclasses.dataclass
class Config:
    hidden: int = 512
    layers: str = "gga"  # g: gated delta rule, a: attention
    H: int = 4           # the recurrence's key heads, value heads and head size
    HV: int = 8
    K: int = 128
    width: int = 4       # of the convolution
    HQ: int = 8          # attention's query heads, kv heads, head size and rotated part
    HK: int = 2
    D: int = 128
    rotary: int = 64
    page: int = 64


class Layer:
    def __init__(self, cfg: Config, kind: str, gen: torch.Generator, device):
        def w(rows, cols):
            return (torch.randn(rows, cols, generator=gen) / math.sqrt(cols)).to(device, BF)
        self.kind, self.norm = kind, torch.ones(cfg.hidden, device=device)
        if kind == "g":
            self.dim = 2 * cfg.H * cfg.K + cfg.HV * cfg.K
            self.w_in = w(self.dim + cfg.HV * cfg.K + 2 * cfg.HV, cfg.hidden)  # q | k | v, gate z, a, b
            self.conv = w(self.dim, cfg.width)
            self.A_log = torch.rand(cfg.HV, generator=gen).mul(15).add(1).log().to(device)
            self.dt_bias = torch.full((cfg.HV,), -3.0, device=device)
            self.out_norm = torch.ones(cfg.K, device=device)
            self.w_out = w(cfg.hidden, cfg.HV * cfg.K)
        else:
            self.w_in = w((cfg.HQ + 2 * cfg.HK) * cfg.D, cfg.hidden)
            self.w_out = w(cfg.hidden, cfg.HQ * cfg.D)


class HybridStack:
    """Weights, and what is kept for `requests` requests of up to `context` tokens each."""

    def __init__(self, cfg: Config = Config(), requests: int = 8, context: int = 1024, seed: int = 0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        self.cfg, self.device, self.requests = cfg, device, requests
        self.layers = [Layer(cfg, kind, gen, device) for kind in cfg.layers]
        self.norm = torch.ones(cfg.hidden, device=device)
        self.inv_freq, self.rope_factor = rope_frequencies(cfg.rotary, device=device)
        ints = dict(dtype=torch.int32, device=device)
        width = -(-context // cfg.page)
        pages = requests * width
        # the paged cache: one table for all attention layers, codes and scales for each
        self.table = torch.full((requests, width), -1, **ints)
        self.free = torch.arange(pages, **ints)
        self.num_free = torch.tensor([pages], **ints)
        self.lens = torch.zeros(requests, **ints)
        self.status = torch.zeros(1, **ints)
        self.rows = torch.arange(requests, **ints)
        for layer in self.layers:
            if layer.kind == "a":
                shape = (pages, cfg.HK, cfg.page, cfg.D)
                layer.cache = [torch.zeros(shape, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)] + \
                              [torch.ones(shape[:2], device=device) for _ in range(2)]
            else:
                layer.state = torch.zeros(requests, cfg.HV, cfg.K, cfg.K, device=device)
                layer.conv_state = torch.zeros(requests, layer.dim, cfg.width - 1, dtype=BF, device=device)

    # ------------------------------------------------------------- serving
    def step(self, x: torch.Tensor, news: List[int]) -> torch.Tensor:
        """x bf16 [T, hidden]: news[n] further tokens of every request n, in order.  Returns [T, hidden]."""
        cfg, T = self.cfg, x.shape[0]
        cu = torch.tensor([0] + news, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(self.device)
        single = all(m == 1 for m in news)
        plan = gdn_paged_plan(self.lens, cu, self.table, self.free, self.num_free, cfg.page, T, dev_status=self.status)
        lens, slots, positions, num_free = plan
        started = self.lens > 0
        h, y = x, None  # the residual stream, and what the last block adds to it
        for layer in self.layers:
            if y is None:
                n, _ = gdn_norm_gate(h, layer.norm)
            else:
                n, h = gdn_norm_gate(y, layer.norm, residual=h)
            u = n @ layer.w_in.T
            if layer.kind == "a":
                qkv = u.view(T, cfg.HQ + 2 * cfg.HK, cfg.D)
                q, k, v = qkv.split([cfg.HQ, cfg.HK, cfg.HK], dim=1)
                q, k = gdn_rope(q, k, positions, self.inv_freq, attention_factor=self.rope_factor)
                gdn_kv8_append(k, v, *layer.cache, slots, dev_status=self.status)
                o = gdn_kv8_attention(q, *layer.cache, self.table, lens, cu_seqlens=None if single else cu, max_q_len=max(news),
                                      dev_status=self.status)
            else:
                o = self._recurrence(layer, u, cu, started, single)
                # the block's own norm, one head a row, gated by a slice of the projection
                z = u[:, layer.dim:layer.dim + cfg.HV * cfg.K].unflatten(1, (cfg.HV, cfg.K))
                o, _ = gdn_norm_gate(o.view(T, cfg.HV, cfg.K), layer.out_norm, z=z)
            y = o.reshape(T, -1) @ layer.w_out.T
        out, _ = gdn_norm_gate(y, self.norm, residual=h)
        self.lens, self.num_free = lens, num_free
        return out

    def _recurrence(self, layer, u, cu, started, single):
        cfg, T = self.cfg, u.shape[0]
        a, b = (t.contiguous() for t in u[:, layer.dim + cfg.HV * cfg.K:].chunk(2, dim=1))
        gates = dict(A_log=layer.A_log, dt_bias=layer.dt_bias)
        if single:
            q, k, v = gdn_conv_decode_pack(u[:, :layer.dim].contiguous(), layer.conv_state, layer.conv, None, self.rows, cfg.H,
                                           cfg.HV, cfg.K, cfg.K, dev_status=self.status)
            return gdn_recurrent_decode(q, k, v, layer.state, self.rows, a=a, b=b, dev_status=self.status, **gates)
        m = gdn_causal_conv1d_fwd(u[:, :layer.dim].T.contiguous(), layer.conv, None, layer.conv_state, cu, cache_indices=self.rows,
                                  has_initial_state=started, dev_status=self.status).T.contiguous()
        q, k, v = m.split([cfg.H * cfg.K, cfg.H * cfg.K, cfg.HV * cfg.K], dim=1)
        q, k, v = (t.contiguous().view(1, T, -1, cfg.K) for t in (q, k, v))
        o, layer.state = gdn_chunk_fwd_gated(q, k, v, a=a.view(1, T, -1), b=b.view(1, T, -1), initial_state=layer.state,
                                             cu_seqlens=cu, num_seqs=self.requests, dev_status=self.status, **gates)
        return o

    # ------------------------------------------------------------ training
    def parameters(self) -> List[torch.Tensor]:
        out = [self.norm]
        for layer in self.layers:
            out += [layer.norm, layer.w_in, layer.w_out] + ([layer.out_norm] if layer.kind == "g" else [])
        return out

    def _plain_attention(self, q, k, v):
        """Causal attention of one sequence in fp32, from elementary operations."""
        cfg, T = self.cfg, q.shape[0]
        k, v = (t.repeat_interleave(cfg.HQ // cfg.HK, dim=1).transpose(0, 1).float() for t in (k, v))
        s = q.transpose(0, 1).float() @ k.transpose(1, 2) / math.sqrt(cfg.D)
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=q.device).triu(1), -math.inf)
        return (s.softmax(-1) @ v).transpose(0, 1).to(BF)

    def forward(self, x: torch.Tensor, lens: Optional[List[int]] = None, save8: bool = False) -> torch.Tensor:
        """Differentiable, for x bf16 [T, hidden] from its beginning (no convolution): one sequence, whose attention has fp32
        logits and weights ([heads, T, T] of them in memory), or packed sequences of the lengths ``lens`` ([T] for one), whose
        attention is ``attention``, with its weights in bf16 (heads of other sizes than 64 and 128: as without lens).  With
        ``save8``, which takes ``attention`` too, the norms and projections keep their inputs for the gradient in 8 bits."""
        cfg, T = self.cfg, x.shape[0]
        kernels = (lens is not None or save8) and cfg.D in (64, 128)
        if lens is None:
            cu, num_seqs, positions = None, None, torch.arange(T, dtype=torch.int32, device=x.device)
        else:
            lens = [int(m) for m in lens]
            if not lens or min(lens) < 0 or sum(lens) != T:
                raise ValueError(f"HybridStack: lens must be lengths that add up to x's {T} tokens, got {lens}")
            cu, num_seqs = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(x.device), len(lens)
            positions = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).to(x.device)
        plain = lambda x, w: x @ w.T  # noqa: E731
        linear = linear8 if save8 else plain
        h, y = x, None
        for layer in self.layers:
            if y is None:
                n, _ = norm_gate(h, layer.norm, save8=save8)
            else:
                n, h = norm_gate(y, layer.norm, residual=h, save8=save8)
            u = linear(n, layer.w_in)
            if layer.kind == "a":
                q, k, v = u.view(T, -1, cfg.D).split([cfg.HQ, cfg.HK, cfg.HK], dim=1)
                q, k = rotary_embedding(q, k, positions, self.inv_freq, attention_factor=self.rope_factor)
                if kernels:
                    if save8:  # it keeps v, and with a view of the projection all of that
                        v = v.contiguous()
                    o = attention(q, k, v, cu_seqlens=cu, dev_status=self.status)
                elif lens is None:
                    o = self._plain_attention(q, k, v)
                else:
                    o = torch.cat([self._plain_attention(*part) for part in zip(*(t.split(lens) for t in (q, k, v)))])
            else:
                q, k, v, z, a, b = u.split([cfg.H * cfg.K, cfg.H * cfg.K, cfg.HV * cfg.K, cfg.HV * cfg.K, cfg.HV, cfg.HV], dim=1)
                q, k, v = (t.contiguous().view(1, T, -1, cfg.K) for t in (q, k, v))
                g = -layer.A_log.exp() * torch.nn.functional.softplus(a.float() + layer.dt_bias)
                o, _ = chunk_gated_delta_rule(q, k, v, g.view(1, T, -1), b.float().sigmoid().view(1, T, -1), output_final_state=False,
                                              cu_seqlens=cu, num_seqs=num_seqs)
                o, _ = norm_gate(o.view(T, cfg.HV, cfg.K), layer.out_norm, z=z.unflatten(1, (cfg.HV, cfg.K)), save8=save8)
            # (the attention keeps o itself, which a plain product shares)
            y = (plain if layer.kind == "a" and kernels else linear)(o.reshape(T, -1), layer.w_out)
        return norm_gate(y, self.norm, residual=h, save8=save8)[0]

    def train_step(self, x: torch.Tensor, target: torch.Tensor, rate: float = 1e-2, lens: Optional[List[int]] = None,
                   save8: bool = False) -> float:
        """One step of gradient descent on the mean square difference from target; returns the loss before it."""
        params = [p.requires_grad_(True) for p in self.parameters()]
        loss = (self.forward(x, lens, save8).float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, g in zip(params, grads):
                p.requires_grad_(False)
                p.sub_((rate * g.float()).to(p.dtype))
        return float(loss.detach())


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300, help="tokens of the longest prompt")
    ap.add_argument("--tokens", type=int, default=16, help="single tokens after the prompts")
    args = ap.parse_args(argv)
    gen = torch.Generator().manual_seed(1)
    news = [max(1, args.prompt * (n + 1) // args.requests) for n in range(args.requests)]
    stack = HybridStack(requests=args.requests, context=args.prompt + args.tokens)
    x = torch.randn(sum(news), stack.cfg.hidden, generator=gen).to(stack.device, BF)
    ends = torch.tensor(news).cumsum(0).to(stack.device) - 1
    x = stack.step(x, news)[ends]
    for _ in range(args.tokens):
        x = stack.step(x, [1] * args.requests)
    print(f"{args.requests} requests, prompts of {news}, {args.tokens} tokens each: contexts {stack.lens.tolist()}, "
          f"free pages {int(stack.num_free)}, status {int(stack.status)}")
    train = HybridStack(seed=2, requests=1)
    x, t = (torch.randn(256, train.cfg.hidden, generator=gen).to(train.device, BF) for _ in range(2))
    print("training, mean square difference:", " ".join(f"{train.train_step(x, t, 0.5):.4f}" for _ in range(5)))
    lens = [100, 1, 155]
    print("packed sequences:", " ".join(f"{train.train_step(x, t, 0.5, lens):.4f}" for _ in range(5)))
    print("inputs kept in 8 bits:", " ".join(f"{train.train_step(x, t, 0.5, lens, True):.4f}" for _ in range(5)))
    print("status", int(train.status))


if __name__ == "__main__":
    main()
