"""gdn_attn_decode_shared against softmax attention in 64 bits.

Tolerance, with A = sum p |v| (the weighted mean of the values' sizes): a
weight rounded to bf16 is off by at most 2^-8 of itself, so the sum by 2^-8 A;
the fp32 scores and exponentials move the weights by less than 2^-11 together;
the result is rounded once, 2^-8 |o|.  The gate multiplies all of it.
"""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def build(B, S, hq, hk, d, page, prefix, tails, seed=0, std=1.5, poison=True, gate=True):
    """Random pages in random order; everything that no sequence owns is NaN or inf."""
    g = torch.Generator().manual_seed(seed)
    npre = -(-prefix // page)
    per = [-(-t // page) for t in tails]
    width = max(per + [0])
    pages = npre + sum(per) + 2
    perm = torch.randperm(pages, generator=g)
    fill = float("nan") if poison else 0.0
    kc = torch.full((pages, page, hk, d), fill, dtype=BF)
    vc = torch.full((pages, page, hk, d), float("inf") if poison else 0.0, dtype=BF)
    tp = torch.full((B, width), -9, dtype=torch.int32)   # entries past a tail's end are never read
    at = npre
    seqs = []

    def put(page_ids, n):
        k = (torch.randn(n, hk, d, generator=g) * std).to(BF)
        v = torch.randn(n, hk, d, generator=g).to(BF)
        for j in range(n):
            kc[page_ids[j // page], j % page] = k[j]
            vc[page_ids[j // page], j % page] = v[j]
        return k, v

    pre = put(perm[:npre], prefix)
    for b in range(B):
        ids = perm[at:at + per[b]]
        at += per[b]
        tp[b, :per[b]] = ids.int()
        seqs.append(put(ids, tails[b]))
    q = torch.randn(B, S, hq, d, generator=g).to(BF)
    gt = torch.randn(B, S, hq, 2 * d, generator=g).to(BF) if gate else None
    return dict(q=q, kc=kc, vc=vc, pp=perm[:npre].int(), prefix=prefix, tp=tp if width else None,
                tl=torch.tensor(tails, dtype=torch.int32) if width else None, pre=pre, seqs=seqs, gate=gt,
                tails=tails)


def reference(x, hk, scale):
    q = x["q"].double()
    B, S, hq, d = q.shape
    G = hq // hk
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    for b in range(B):
        k = torch.cat([x["pre"][0], x["seqs"][b][0]]).double()
        v = torch.cat([x["pre"][1], x["seqs"][b][1]]).double()
        for i in range(S):
            n = x["prefix"] + max(0, x["tails"][b] - S + 1 + i)
            if n == 0:
                continue
            for h in range(hq):
                p = torch.softmax(k[:n, h // G] @ q[b, i, h] * scale, 0)
                out[b, i, h] = p @ v[:n, h // G]
                size[b, i, h] = p @ v[:n, h // G].abs()
    if x["gate"] is not None:
        f = torch.sigmoid(x["gate"][..., d:].double())
        out, size = out * f, size * f
    return out, size


def call(dims, x, ws=None):
    B, S, hq, d = x["q"].shape
    dev = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in x.items() if k not in ("pre", "seqs")}
    if ws is None:
        ws = torch.full((gdn.gdn_attn_decode_shared_workspace_bytes(dims, B, S),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((B, S, hq, d), float("nan"), dtype=BF, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    gate = dev["gate"][..., d:] if dev["gate"] is not None else None
    gdn.gdn_attn_decode_shared(dims, dev["q"], dev["kc"], dev["vc"], dev["pp"], x["prefix"], dev["tp"], dev["tl"],
                               out, ws, gate=gate, device_status=st)
    return out, gdn.gdn_read_device_status(st)


def check(dims, x):
    out, st = call(dims, x)
    assert st == 0
    ref, size = reference(x, dims.h_kv, dims.scale or dims.d ** -0.5)
    tol = (2.0 ** -8 + 2.0 ** -11) * size + 2.0 ** -8 * ref.abs()
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() - tol
    assert (bad <= 0).all(), (float(bad.max()), int((bad > 0).sum()))
    return out


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,S,hq,hk,page,prefix,tails", [
    (1, 1, 1, 1, 16, 0, [1]),                        # one token in all
    (1, 1, 2, 1, 16, 1, [0]),                        # one token of the prefix
    (2, 1, 4, 2, 32, 0, [0, 3]),                     # a row that sees nothing
    (3, 4, 4, 1, 16, 0, [2, 4, 7]),                  # rows of a sequence that see nothing
    (1, 1, 16, 2, 64, 64, [64]),                     # whole tiles
    (5, 1, 6, 2, 64, 131, [1, 63, 64, 65, 130]),     # pages that end inside a tile, odd group
    (4, 8, 8, 1, 16, 77, [8, 9, 40, 3]),             # eight tokens each, one tail shorter than they
    (2, 3, 10, 2, 128, 300, [129, 257]),
    (3, 1, 7, 7, 256, 513, [300, 0, 255]),           # no sharing of heads
])
def test_matches_the_definition(d, B, S, hq, hk, page, prefix, tails):
    dims = gdn.make_attn_dims(h_q=hq, h_kv=hk, d=d, rot=0)
    check(dims, build(B, S, hq, hk, d, page, prefix, tails, seed=B + d))


@pytest.mark.parametrize("d,B,S,hq,hk,prefix,hi", [
    (128, 40, 1, 8, 1, 700, 90), (256, 70, 1, 4, 2, 1500, 40), (64, 33, 4, 12, 2, 900, 30), (256, 17, 8, 16, 1, 333, 20),
    (128, 1, 1, 2, 1, 9000, 50), (256, 3, 1, 128, 1, 200, 70), (64, 130, 1, 2, 2, 100, 260)])
def test_many_rows_and_long_prefixes(d, B, S, hq, hk, prefix, hi):
    # several tiles of 128 rows, and ranges of keys split over the GPU
    g = torch.Generator().manual_seed(B)
    tails = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    dims = gdn.make_attn_dims(h_q=hq, h_kv=hk, d=d, rot=0)
    check(dims, build(B, S, hq, hk, d, 32, prefix, tails, seed=d))


def test_no_prefix_no_tails_and_empty():
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=64, rot=0)
    x = build(3, 1, 4, 2, 64, 16, 50, [0, 0, 0])     # no tails at all: no tables
    assert x["tp"] is None
    check(dims, x)
    x = build(2, 2, 4, 2, 64, 16, 0, [0, 0], gate=False)
    out, st = call(dims, x)
    assert st == 0 and (out == 0).all()


def test_peaked_and_flat_maps_and_extreme_scores():
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=128, rot=0)
    # scores of several hundred: one key takes all; the running maximum jumps late
    x = build(2, 1, 4, 2, 128, 16, 400, [37, 90], std=60.0)
    check(dims, x)
    # all keys alike
    x = build(2, 1, 4, 2, 128, 16, 400, [37, 90], std=0.0)
    check(dims, x)
    # a custom scale
    check(gdn.make_attn_dims(h_q=4, h_kv=2, d=128, rot=0, scale=0.5),
          build(2, 1, 4, 2, 128, 16, 100, [5, 6], std=0.3))


def test_bad_pages_and_lengths_are_reported_and_stay_in_their_sequence():
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=64, rot=0)
    x = build(4, 1, 4, 2, 64, 16, 40, [20, 33, 16, 7])
    good, st = call(dims, x)
    assert st == 0
    for b, j, v in ((1, 2, 1 << 30), (1, 0, -1), (1, 1, x["kc"].shape[0])):
        y = dict(x, tp=x["tp"].clone())
        y["tp"][b, j] = v
        out, st = call(dims, y)
        assert st == gdn.GDN_ERR_DEVICE_BOUNDS
        assert torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
    for n in (-1, 16 * x["tp"].shape[1] + 1, 1 << 30):
        y = dict(x, tl=x["tl"].clone())
        y["tl"][2] = n
        _, st = call(dims, y)
        assert st == gdn.GDN_ERR_DEVICE_BOUNDS
    y = dict(x, pp=x["pp"].clone())
    y["pp"][1] = -5
    assert call(dims, y)[1] == gdn.GDN_ERR_DEVICE_BOUNDS


def test_equal_calls_give_equal_bits_on_any_stream_and_in_graphs():
    dims = gdn.make_attn_dims(h_q=8, h_kv=2, d=128, rot=0)
    x = build(19, 2, 8, 2, 128, 16, 777, [(i * 13) % 90 + 2 for i in range(19)])
    a, _ = call(dims, x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b, _ = call(dims, x)
    s.synchronize()
    assert torch.equal(a, b)
    # a captured step stays valid while the tails grow
    dev = {k: v.to(DEV) for k, v in x.items() if isinstance(v, torch.Tensor)}
    ws = torch.empty(gdn.gdn_attn_decode_shared_workspace_bytes(dims, 19, 2), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(a)
    tl = torch.full_like(dev["tl"], 2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_attn_decode_shared(dims, dev["q"], dev["kc"], dev["vc"], dev["pp"], 777, dev["tp"], tl, out, ws,
                                   gate=dev["gate"][..., 128:])
    tl.copy_(dev["tl"])
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)


def test_offsets_past_32_bits():
    # a cache of 2^31 + elements: pages beyond 4 GB hold the data
    hk, d, page = 1, 256, 256
    pages = (1 << 32) // (page * hk * d) + 40
    dims = gdn.make_attn_dims(h_q=4, h_kv=hk, d=d, rot=0)
    x = build(2, 1, 4, hk, d, page, 600, [300, 5], poison=False)
    n = x["kc"].shape[0]
    out, _ = call(dims, x)
    kc = torch.empty(pages, page, hk, d, dtype=BF, device=DEV)
    vc = torch.empty(pages, page, hk, d, dtype=BF, device=DEV)
    kc[-n:], vc[-n:] = x["kc"].to(DEV), x["vc"].to(DEV)
    y = dict(x, kc=kc, vc=vc, pp=x["pp"] + pages - n, tp=x["tp"] + pages - n)
    far, st = call(dims, y)
    assert st == 0 and torch.equal(far, out)
