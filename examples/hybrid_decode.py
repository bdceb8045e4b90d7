"""A decode step of a small hybrid model, with every block this library has.

One group of layers: a Gated DeltaNet layer and a gated-attention layer, each
followed by a mixture-of-experts block, for a batch of sequences that share a
prompt.  The prompt is read once: its Gated DeltaNet state is copied to every
sequence, its keys and values stay in shared pages of the cache.  Then every
sequence decodes tokens of its own; the attention reads the prompt's pages
once for the batch and each sequence's own pages after them.

    python examples/hybrid_decode.py

prints the largest difference between the batch and one of its sequences
decoded alone, with the prompt in its own pages instead of shared ones.
Random weights and inputs; a model's norms and projections around the blocks
are plain torch operations.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_06_gb300 as gdn  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
PAGE, ROT = 16, 64


def rms(x, eps=1e-6):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)).to(BF)


class Block:
    """Weights of the two layers and their expert blocks."""

    def __init__(self, hidden=512, h_k=4, h_v=8, h_q=8, h_kv=2, d=128, experts=32, inter=128, top_k=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std=None: (torch.randn(*s, generator=g, device="cuda") *
                                  (s[-1] ** -0.5 if std is None else std)).to(BF)
        self.hidden = hidden
        self.gdn = gdn.make_dims(h_k=h_k, h_v=h_v)
        self.attn = gdn.make_attn_dims(h_q=h_q, h_kv=h_kv, d=d, rot=ROT, n_axes=3)
        self.moe = gdn.make_moe_dims(hidden=hidden, inter=inter, experts=experts, top_k=top_k, shared_inter=inter)
        cc = 2 * h_k * 128 + h_v * 128
        self.w_in, self.w_out = r(gdn.in_proj_features(self.gdn), hidden), r(hidden, h_v * 128)
        self.cc, self.conv_w = cc, r(cc, 4, std=0.5)
        self.A_log = torch.rand(h_v, generator=g, device="cuda")
        self.dt_bias, self.gdn_norm = torch.zeros(h_v, device="cuda"), torch.ones(128, device="cuda")
        # the attention projection: query heads with their gates beside them, keys, values
        self.w_q, self.w_kv, self.w_o = r(h_q * 2 * d, hidden), r(2 * h_kv * d, hidden), r(hidden, h_q * d)
        self.q_norm, self.k_norm = torch.ones(d, device="cuda"), torch.ones(d, device="cuda")
        self.inv_freq = torch.tensor([1e7 ** (-2 * i / ROT) for i in range(ROT // 2)], dtype=torch.float64, device="cuda")
        self.axis = torch.tensor([i % 3 for i in range(ROT // 2)], dtype=I32, device="cuda")   # time, row, column in turn
        self.experts = [dict(w_router=r(experts, hidden), w_gate_up=r(experts, 2 * inter, hidden),
                             w_down=r(experts, hidden, inter), w_shared_gate_up=r(2 * inter, hidden),
                             w_shared_down=r(hidden, inter), w_shared_gate=r(hidden)) for _ in range(2)]


class Sequences:
    """The states of a batch: Gated DeltaNet states, and pages of one cache."""

    def __init__(self, m: Block, batch, prefix, tail):
        d = m.attn.d
        self.n_prefix, self.per = -(-prefix // PAGE), -(-tail // PAGE)
        pages = self.n_prefix + batch * self.per
        self.k = torch.zeros(pages, PAGE, m.attn.h_kv, d, dtype=BF, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.conv = torch.zeros(batch, 3, m.cc, device="cuda")
        self.ssm = torch.zeros(batch, m.gdn.h_v, 128, 128, device="cuda")
        self.prefix_pages = torch.arange(self.n_prefix, dtype=I32, device="cuda")
        self.tail_pages = (torch.arange(batch * self.per, dtype=I32, device="cuda") + self.n_prefix).view(batch, self.per)
        self.tail_len = torch.zeros(batch, dtype=I32, device="cuda")
        self.prefix = 0
        self.status = torch.zeros(1, dtype=I32, device="cuda")


def step(m: Block, s: Sequences, x, pos):
    """x [B, S, hidden] at positions pos [3, B, S] -> [B, S, hidden]; S <= 8 new
    tokens per sequence."""
    B, S, H = x.shape
    a, T = m.attn, B * S

    def mix(x, e):
        y = torch.empty_like(x)
        for lo in range(0, T, 64):       # the expert call takes up to 64 tokens
            part = rms(x[lo:lo + 64]).contiguous()
            ws = torch.empty(gdn.gdn_moe_step_workspace_bytes(m.moe, part.shape[0]), dtype=torch.uint8, device="cuda")
            gdn.gdn_moe_step(m.moe, part, e["w_router"], e["w_gate_up"], e["w_down"], y[lo:lo + 64], ws,
                             w_shared_gate_up=e["w_shared_gate_up"], w_shared_down=e["w_shared_down"],
                             w_shared_gate=e["w_shared_gate"], device_status=s.status)
        return x + y

    x = x.reshape(T, H)
    # the Gated DeltaNet layer
    g = m.gdn
    qkv, z = torch.empty(T, m.cc, dtype=BF, device="cuda"), torch.empty(T, g.h_v, 128, dtype=BF, device="cuda")
    al, be = torch.empty(T, g.h_v, dtype=BF, device="cuda"), torch.empty(T, g.h_v, dtype=BF, device="cuda")
    gdn.gdn_in_proj(g, H, rms(x), m.w_in, qkv, z, al, be)
    o = torch.empty(B, S, g.h_v, 128, dtype=BF, device="cuda")
    gdn.gdn_decode_multi(g, qkv, z, al, be, m.A_log, m.dt_bias, m.conv_w, m.gdn_norm, None, B, s.conv, s.ssm, o, S,
                         device_status=s.status)
    y = torch.empty(T, H, dtype=BF, device="cuda")
    gdn.gdn_out_proj(g, H, o.view(T, g.h_v, 128), m.w_out, y)
    x = mix(x + y, m.experts[0])
    # the gated-attention layer: the new keys and values into the tails' pages, then all
    # of a sequence's keys
    xn = rms(x)
    qg = (xn @ m.w_q.t()).view(T, a.h_q, 2 * a.d)
    kv = (xn @ m.w_kv.t()).view(T, 2, a.h_kv, a.d)
    at = s.tail_len[:, None] + torch.arange(S, device="cuda")                       # place in the tail
    slot = torch.gather(s.tail_pages, 1, (at // PAGE).long()) * PAGE + at % PAGE
    q = torch.empty(B, S, a.h_q, a.d, dtype=BF, device="cuda")
    gdn.gdn_attn_prep(a, qg[..., :a.d], kv[:, 0], kv[:, 1], m.q_norm, m.k_norm, m.inv_freq, m.axis,
                      pos.reshape(3, T).contiguous(), q, s.k, s.v, slot=slot.reshape(T).to(I32).contiguous(),
                      device_status=s.status)
    s.tail_len += S
    out = torch.empty_like(q)
    ws = torch.empty(gdn.gdn_attn_decode_shared_workspace_bytes(a, B, S), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_decode_shared(a, q, s.k, s.v, s.prefix_pages, s.prefix, s.tail_pages, s.tail_len, out, ws,
                               gate=qg[..., a.d:], device_status=s.status)
    x = mix(x + out.view(T, a.h_q * a.d) @ m.w_o.t(), m.experts[1])
    return x.view(B, S, H)


def read_prompt(m, s, x):
    """The prompt [L, hidden] through the block, 8 tokens a step, as the tail of a
    batch of one."""
    for i in range(0, x.shape[0], 8):
        part = x[None, i:i + 8].contiguous()
        pos = (i + torch.arange(part.shape[1], device="cuda")).expand(3, 1, -1).to(I32)
        step(m, s, part, pos)


def main(batch=6, prompt=200, tokens=5, verbose=True):
    m = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompt_x = torch.randn(prompt, m.hidden, generator=g, device="cuda").to(BF)
    own_x = torch.randn(tokens, batch, m.hidden, generator=g, device="cuda").to(BF)

    alone = Sequences(m, 1, 0, prompt + tokens)       # the prompt in its own pages
    read_prompt(m, alone, prompt_x)
    # the batch: one prompt in shared pages, its state copied to every sequence
    many = Sequences(m, batch, prompt, tokens)
    many.prefix = prompt
    many.k[:many.n_prefix], many.v[:many.n_prefix] = alone.k[:many.n_prefix], alone.v[:many.n_prefix]
    zero = torch.zeros(batch, dtype=I32, device="cuda")
    gdn.gdn_state_copy(m.gdn, alone.conv, alone.ssm, many.conv, many.ssm, src_slot=zero, n=batch)

    worst = 0.0
    for t in range(tokens):
        pos = torch.full((3, batch, 1), prompt + t, dtype=I32, device="cuda")
        y = step(m, many, own_x[t][:, None], pos)
        one = step(m, alone, own_x[t][:1, None].contiguous(), pos[:, :1].contiguous())
        worst = max(worst, float((y[:1].float() - one.float()).abs().max() / one.float().abs().max()))
    assert gdn.gdn_read_device_status(many.status) == 0 and gdn.gdn_read_device_status(alone.status) == 0
    if verbose:
        print(f"{batch} sequences after a shared prompt of {prompt} tokens, {tokens} steps: sequence 0 differs from "
              f"itself alone by at most {worst:.1e} of its largest output")
    return worst


if __name__ == "__main__":
    main()
