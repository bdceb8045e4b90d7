"""What a forked, trimmed and compacted pool serves, held to what its sequences are.

The first layer's keys and values depend on the tokens alone, so a continuation's rows, read
through its table, are the bits of the sequence held alone.  Every layer's attention outputs
are held to softmax attention in 64 bits, over the rows of the sequence alone (first layer)
or over the continuation's own (both), with test_attn_kv4_gpu's tolerance.  The same tolerance
tells a sequence that lacks its last token or has other rows in a page apart."""
import os
import sys

import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(m, c, seq, layer, n):
    """The first n rows of a sequence, K and V [n, h, d] fp32, through its table."""
    page, at = c.pool.page, torch.arange(n, device="cuda")
    slot = (c.table[seq].long()[at // page] * page + at % page).to(torch.int32)
    k, v = (torch.empty(n, m.dims.h_kv, m.dims.d, device="cuda") for _ in range(2))
    gdn.gdn_kv4_load(m.dims, c.kv[layer], k, v, slot=slot, device_status=c.status)
    return k, v


def worst(m, q, gate, out, k, v):
    """Largest error of out [h_q, d] in units of the tolerance, over the rows k and v."""
    G, d = m.dims.h_q // m.dims.h_kv, m.dims.d
    k, v = (x.double().repeat_interleave(G, 1) for x in (k, v))
    most = v.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
    p = torch.softmax(torch.einsum("nhd,hd->hn", k, q.double()) * d ** -0.5, -1)
    f = torch.sigmoid(gate.double())
    want = torch.einsum("hn,nhd->hd", p, v) * f
    size = torch.einsum("hn,nhd->hd", p, v.abs() + 2 ** -6 * most) * f
    return ((out.double() - want).abs() / (2 ** -8 * want.abs() + 2 ** -10 * size + 1e-30)).max().item()


@pytest.mark.parametrize("prompt,tokens,children", [(77, 6, 3), (16, 3, 1), (5, 2, 12), (301, 4, 7), (40, 2, 2)])
def test_rows_and_attention_are_the_sequences(prompt, tokens, children):
    import paged_decode as pd
    m = pd.Model()
    g = torch.Generator(device="cuda").manual_seed(prompt)
    rand = lambda *s: torch.randn(*s, m.hidden, generator=g, device="cuda").to(BF)   # noqa: E731
    first, other, own, drafts = rand(prompt), rand(prompt // 2 + 3), rand(tokens, children), rand(children, 3)
    c = pd.Cache(m, children + 2, 200)
    pd.read(m, c, 0, first)
    pd.read(m, c, 1, other)
    kids = list(range(2, 2 + children))
    gdn.gdn_pages_fork(c.pool, c.caches, c.i32([0] * children), c.i32(kids), c.ws, device_status=c.status)
    alone = []
    for i in range(children):
        a = pd.Cache(m, 1, 64)
        pd.read(m, a, 0, first)
        for t in range(tokens):
            pd.step(m, a, [0], own[t, i][None, None])
        alone.append((a, *rows(m, a, 0, 0, prompt + tokens)))
        assert a.lens.tolist() == [prompt + tokens]
    told = []
    for t in range(tokens):
        heads, n = [], prompt + t + 1
        pd.step(m, c, kids, own[t][:, None], heads)
        assert c.lens[2:].tolist() == [n] * children
        for i, s in enumerate(kids):
            q, gate, out = (x[i, 0] for x in heads[0])
            _, k, v = alone[i]
            assert worst(m, q, gate, out, k[:n], v[:n]) <= 1
            for layer, x in enumerate(heads):
                assert worst(m, *(y[i, 0] for y in x), *rows(m, c, s, layer, n)) <= 1
            # mistakes, in what it is held to: no last token, other rows in a page
            told.append(worst(m, q, gate, out, k[:n - 1], v[:n - 1]) if n > 1 else 2)
            if n >= 16:
                k, v = k[:n].clone(), v[:n].clone()
                wrong = torch.randn(16, m.dims.h_kv, m.dims.d, generator=g, device="cuda")
                k[:16], v[:16] = wrong, wrong.flip(0)
                told.append(worst(m, q, gate, out, k, v))
        before = c.lens[2:].clone()
        pd.step(m, c, kids, drafts)
        gdn.gdn_pages_trim(c.pool, c.caches, before, c.ws, seq=c.i32(kids), device_status=c.status)
        if t == tokens // 2:
            gdn.gdn_pages_free(c.pool, c.i32([0, 1]), c.ws, device_status=c.status)
            gdn.gdn_pages_compact(c.pool, c.caches, c.ws, device_status=c.status)
    assert min(told) > 1, min(told)
    for i, s in enumerate(kids):
        for got, want in zip(rows(m, c, s, 0, prompt + tokens), alone[i][1:]):
            assert torch.equal(got, want)
    assert gdn.gdn_read_device_status(c.status) == 0
