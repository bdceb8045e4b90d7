"""Serving sequences from one pool of cache pages, held in 4 bits.

Two gated-attention layers whose caches follow the same page tables.  Prompts
are read in, one of them is forked into several continuations that share its
whole pages, tokens are drafted and partly taken back, a continuation is
dropped and the pool is drawn together, all between decode steps of the batch:

    extend (new tokens' rows) -> norms and positions -> rows into the 4-bit
    cache -> attention through the tables

    python examples/paged_decode.py

prints the largest difference between a continuation's attention outputs and those
of the same sequence decoded alone, in a pool of its own, without any of that (the
layers' outputs are mostly their inputs, which would hide one).  Random weights
and inputs; a model's norms and projections around the layers are plain torch
operations.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_06_gb300 as gdn  # noqa: E402

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
ROT, LAYERS = 64, 2


def rms(x, eps=1e-6):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)).to(BF)


class Model:
    def __init__(self, hidden=512, h_q=8, h_kv=2, d=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).to(BF)   # noqa: E731
        self.hidden, self.dims = hidden, gdn.make_attn_dims(h_q=h_q, h_kv=h_kv, d=d, rot=ROT)
        self.layers = [dict(w_q=r(h_q * 2 * d, hidden), w_kv=r(2 * h_kv * d, hidden), w_o=r(hidden, h_q * d))
                       for _ in range(LAYERS)]
        self.q_norm, self.k_norm = torch.ones(d, device="cuda"), torch.ones(d, device="cuda")
        self.inv_freq = torch.tensor([1e7 ** (-2 * i / ROT) for i in range(ROT // 2)], dtype=torch.float64, device="cuda")


class Cache:
    """A pool of pages and the caches that follow its tables."""

    def __init__(self, m: Model, seqs, pages, page=16, width=64):
        self.refs = torch.zeros(pages, dtype=I32, device="cuda")
        self.table = torch.full((seqs, width), -1, dtype=I32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=I32, device="cuda")
        self.pool = gdn.make_page_pool(self.refs, self.table, self.lens, page)
        self.kv = [torch.zeros(pages, m.dims.h_kv, page // 16, 18 * m.dims.d, dtype=U8, device="cuda")
                   for _ in range(LAYERS)]
        self.caches = gdn.make_page_caches(self.kv)
        self.ws = torch.empty(gdn.gdn_pages_workspace_bytes(self.pool), dtype=U8, device="cuda")
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def i32(self, values):
        return torch.tensor(values, dtype=I32, device="cuda")


def step(m: Model, c: Cache, seqs, x, heads=None):
    """x [n, S, hidden]: S new tokens (at most 8) of the sequences `seqs` -> [n, S, hidden].  The
    list `heads` takes each layer's queries, gates and attention outputs, [n, S, h_q, d] all."""
    n, S, H = x.shape
    a, T = m.dims, n * S
    seq = c.i32(seqs)
    slot = torch.empty(n, S, dtype=I32, device="cuda")
    pos = (c.lens[seq.long()][:, None] + torch.arange(S, device="cuda")).to(I32).view(1, T)
    gdn.gdn_pages_extend(c.pool, slot, c.ws, seq=seq, device_status=c.status)
    table, lens = c.table[seq.long()].contiguous(), c.lens[seq.long()].contiguous()
    ws = torch.empty(gdn.gdn_attn_decode_kv4_workspace_bytes(a, n, S), dtype=U8, device="cuda")
    x = x.reshape(T, H)
    for w, cache in zip(m.layers, c.kv):
        xn = rms(x)
        qg = (xn @ w["w_q"].t()).view(T, a.h_q, 2 * a.d)
        kv = (xn @ w["w_kv"].t()).view(T, 2, a.h_kv, a.d)
        q, k = torch.empty(n, S, a.h_q, a.d, dtype=BF, device="cuda"), torch.empty(T, a.h_kv, a.d, dtype=BF, device="cuda")
        gdn.gdn_attn_prep(a, qg[..., :a.d], kv[:, 0], None, m.q_norm, m.k_norm, m.inv_freq, None, pos, q, k, None)
        gdn.gdn_kv4_store(a, k, kv[:, 1], cache, slot=slot.view(T), device_status=c.status)
        out = torch.empty_like(q)
        gdn.gdn_attn_decode_kv4(a, q, cache, table, lens, out, ws, gate=qg[..., a.d:], device_status=c.status)
        if heads is not None:
            heads.append((q, qg[..., a.d:].view(n, S, a.h_q, a.d), out))
        x = x + out.view(T, a.h_q * a.d) @ w["w_o"].t()
    return x.view(n, S, H)


def read(m, c, s, x):
    """A prompt [L, hidden] as sequence s, 8 tokens a step."""
    for i in range(0, x.shape[0], 8):
        step(m, c, [s], x[None, i:i + 8].contiguous())


def main(prompt=77, tokens=6, children=3, verbose=True):
    m = Model()
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, m.hidden, generator=g, device="cuda").to(BF)   # noqa: E731
    first, other = rand(prompt), rand(prompt // 2 + 3)
    own = rand(tokens, children)                       # [step][child]: what each child decodes
    drafts = rand(children, 3)

    c = Cache(m, children + 2, 200)
    read(m, c, 0, first)
    read(m, c, 1, other)
    kids = list(range(2, 2 + children))
    gdn.gdn_pages_fork(c.pool, c.caches, c.i32([0] * children), c.i32(kids), c.ws, device_status=c.status)
    got = []
    for t in range(tokens):
        got.append([])
        step(m, c, kids, own[t][:, None], got[t])
        before = c.lens[2:].clone()
        step(m, c, kids, drafts)                       # three drafted tokens, none of them kept
        gdn.gdn_pages_trim(c.pool, c.caches, before, c.ws, seq=c.i32(kids), device_status=c.status)
        if t == tokens // 2:                           # the other sequence goes, and the holes with it
            gdn.gdn_pages_free(c.pool, c.i32([0, 1]), c.ws, device_status=c.status)
            gdn.gdn_pages_compact(c.pool, c.caches, c.ws, device_status=c.status)
    assert gdn.gdn_read_device_status(c.status) == 0
    assert int((c.refs > 0).sum()) == len(set(c.table[c.table >= 0].tolist()))

    worst = 0.0
    for i in range(children):                          # each child again, alone
        a = Cache(m, 1, 64)
        read(m, a, 0, first)
        for t in range(tokens):
            heads = []
            step(m, a, [0], own[t, i][None, None], heads)
            for (_, _, y), (_, _, z) in zip(heads, got[t]):
                worst = max(worst, float((z[i].float() - y[0].float()).abs().max() / y.float().abs().max()))
        assert gdn.gdn_read_device_status(a.status) == 0
    if verbose:
        print(f"{children} continuations of a prompt of {prompt} tokens, {tokens} steps each: their attention differs from "
              f"the same sequences' alone by at most {worst:.1e} of its largest output")
    return worst


if __name__ == "__main__":
    main()
