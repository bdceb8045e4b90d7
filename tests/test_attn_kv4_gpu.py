"""gdn_attn_decode_kv4 against softmax attention in 64 bits over the values that the
cache stands for.

Tolerance, with A = sum p |v|: a weight times its token's scale is rounded to fp16, off by
at most 2^-11 of itself, so the sum by 2^-11 A; scores and exponentials move the
weights by less than 2^-11 together (a group's two products lose 2^-16 scale max |q| M at most,
as below: with |q| to 4 and M to 6 under 2^-12 of a weight for d = 256); the result is rounded once, 2^-8 |o|.  The gate multiplies
all of it.  Codes meet the weights as 0 .. 15 and 8 times the weights are taken off, both in
fp32: a sum passes through 8 scales (M, the largest magnitude that a group holds) times
its weights.  A tensor-core product adds 17 terms, 16 tokens' and the sum so far.  It cuts each
off below a step, 2^-25 of the power of two of the largest; a code below 2^-14 counts as 2^-14
there, which for the smaller of the two places that codes have is 16 p M, and a step of 2^-21 p M.
The largest token's term ends above that step, so 16 terms lose at most 2^-17 p M in a product,
with the largest p: over the units, 2^-17 sum p M.  Where the sum so far is the largest, steps are
2^-24 of it: units come in pairs, with S and T = sum p M of their own, so twice 17 * 2^-24 (S + T).
The 8s are whole numbers times the weights themselves, at S, then S + T: as much again at most.
In all 2^-17 (1 + 0.27 + 0.27) < 2^-16 sum p M."""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
import kv4_util as kv4

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def build(B, S, hq, hk, d, page, lens, seed=0, std=1.5, gate=True, fill=255, spare=2, width=None):
    """Random pages in random order; every byte that no token owns is `fill` (255: NaN scales)."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-max(n, 0) // page) for n in lens]
    width = max(per + [0]) if width is None else width
    pages = sum(per) + spare
    perm = torch.randperm(pages, generator=g)
    dims = gdn.make_attn_dims(h_q=hq, h_kv=hk, d=d, rot=0)
    cache = torch.full((pages, hk, page // 16, 18 * d), fill, dtype=torch.uint8, device=DEV)
    table = torch.full((B, width), -9, dtype=torch.int32)   # entries past a sequence's end are never read
    at, slot = 0, []
    for b in range(B):
        ids = perm[at:at + per[b]]
        at += per[b]
        table[b, :per[b]] = ids.int()
        n = torch.arange(lens[b])
        slot.append(ids[n // page] * page + n % page if lens[b] else n)
    slot = torch.cat(slot).to(torch.int32)
    k = (torch.randn(len(slot), hk, d, generator=g) * std).to(BF)
    v = torch.randn(len(slot), hk, d, generator=g).to(BF)
    if len(slot):
        gdn.gdn_kv4_store(dims, k.to(DEV), v.to(DEV), cache, slot=slot.to(DEV))
    q = torch.randn(B, S, hq, d, generator=g).to(BF)
    gt = torch.randn(B, S, hq, 2 * d, generator=g).to(BF) if gate else None
    return dict(dims=dims, q=q.to(DEV), cache=cache, table=table.to(DEV) if width else None,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), gate=gt.to(DEV) if gate else None,
                slot=slot, host=lens)


def values(x):
    """K and V that the cache stands for, [tokens, h, d] in 64 bits, by the definition."""
    if not len(x["slot"]):
        return None, None
    return [t.to(DEV) for t in kv4.load(x["cache"], x["slot"].numpy())]


def reference(x, scale=None):
    k, v = values(x)
    q = x["q"].double()
    B, S, hq, d = q.shape
    G = hq // x["dims"].h_kv
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    if k is not None:
        most = v.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
    at = 0
    for b, n_all in enumerate(x["host"]):
        for i in range(S):
            n = n_all - S + 1 + i
            if n <= 0:
                continue
            kk, vv = k[at:at + n].repeat_interleave(G, 1), v[at:at + n].repeat_interleave(G, 1)
            p = torch.softmax(torch.einsum("nhd,hd->hn", kk, q[b, i]) * (scale or d ** -0.5), -1)
            out[b, i] = torch.einsum("hn,nhd->hd", p, vv)
            # (in units of the tolerance of a weight, 2^-10 with the scores' share)
            size[b, i] = torch.einsum("hn,nhd->hd", p, vv.abs() + 2 ** -6 * most[at:at + n].repeat_interleave(G, 1))
        at += n_all
    if x["gate"] is not None:
        f = torch.sigmoid(x["gate"][..., d:].double())
        out, size = out * f, size * f
    return out, size


def call(x, ws=None, status=None):
    B, S, hq, d = x["q"].shape
    if ws is None:
        n = gdn.gdn_attn_decode_kv4_workspace_bytes(x["dims"], B, S)
        ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((B, S, hq, d), float("nan"), dtype=BF, device=DEV)
    gdn.gdn_attn_decode_kv4(x["dims"], x["q"], x["cache"], x["table"], x["lens"], out, ws,
                            gate=x["gate"][..., d:] if x["gate"] is not None else None, device_status=status)
    return out


def check(x, scale=None):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = call(x, status=status)
    assert gdn.gdn_read_device_status(status) == 0
    want, size = reference(x, scale)
    tol = 2 ** -8 * want.abs() + 2 ** -10 * size + 1e-30
    worst = ((got.double() - want).abs() / tol).max().item()
    assert worst <= 1, worst
    return got


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,S", [(8, 1, 1), (2, 2, 1), (16, 2, 1), (10, 2, 3), (16, 2, 2), (32, 2, 5), (17, 1, 7)])
def test_heads_and_steps(d, hq, hk, S):
    check(build(3, S, hq, hk, d, 32, [S + 3, 70, 161], seed=d + S))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_and_lengths(page):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 255, 257, 600]
    check(build(len(lens), 1, 8, 2, 128, page, lens, seed=page))


@pytest.mark.parametrize("lens", [[0], [1], [2], [16], [33], [0, 0, 0], [3, 0, 1, 0, 2]])
@pytest.mark.parametrize("S", [1, 4])
def test_queries_that_see_little_or_nothing(lens, S):
    x = build(len(lens), S, 4, 1, 64, 16, lens, seed=S)
    got = check(x)
    for b, n in enumerate(lens):
        for i in range(S):
            if n - S + 1 + i <= 0:
                assert (got[b, i] == 0).all()


def test_no_tables_at_all():
    x = build(2, 1, 4, 1, 64, 16, [0, 0], seed=1)
    assert x["table"] is None and (call(x) == 0).all()


@pytest.mark.parametrize("d,hk", [(256, 2), (128, 8), (64, 1)])
def test_long_sequences_in_many_shares(d, hk):
    check(build(2, 1, 8 * hk, hk, d, 64, [9001, 5000], seed=3))


@pytest.mark.parametrize("d,hk,S", [(256, 2, 2), (128, 1, 4), (64, 2, 3)])
def test_long_sequences_with_more_than_eight_rows(d, hk, S):
    check(build(2, S, 16 // S * hk, hk, d, 16, [6003, 2990], seed=13))


def test_many_sequences():
    g = torch.Generator().manual_seed(0)
    check(build(300, 1, 8, 1, 128, 16, torch.randint(0, 120, (300,), generator=g).tolist(), seed=4))


def test_most_sequences_and_rows():
    g = torch.Generator().manual_seed(0)
    check(build(1024, 1, 2, 1, 64, 16, torch.randint(0, 40, (1024,), generator=g).tolist(), seed=4, gate=False))
    check(build(2, 8, 16, 1, 64, 16, [200, 9], seed=5))


def test_peaked_and_growing_scores():
    # keys that grow along the sequence: the largest score so far moves again and again
    x = build(1, 1, 8, 1, 128, 32, [700], seed=6, gate=False)
    n = torch.arange(700)
    k = torch.randn(700, 1, 128, generator=torch.Generator().manual_seed(5)) * (0.02 * n[:, None, None])
    gdn.gdn_kv4_store(x["dims"], k.to(BF).to(DEV), None, x["cache"], slot=x["slot"].to(DEV))
    check(x)


@pytest.mark.parametrize("d,G,S", [(64, 1, 1), (128, 4, 1), (256, 2, 1), (64, 8, 2), (128, 4, 4), (256, 16, 1)])
@pytest.mark.parametrize("ahead", [4.0, 7.0, 10.0])
def test_small_sums_next_to_a_large_weight(d, G, S, ahead):
    # one token takes nearly all the weight and is zero but for a large value in each group:
    # elsewhere the outputs are the others' small sums
    n = 48
    x = build(1, S, G, 1, d, 16, [n], seed=d + G, std=0.5, gate=False)
    g = torch.Generator().manual_seed(14)
    u = torch.randn(d, generator=g)
    x["q"] = (u + 0.02 * torch.randn(1, S, G, d, generator=g)).to(BF).to(DEV)
    k, v = 0.05 * torch.randn(n, 1, d, generator=g), torch.randn(n, 1, d, generator=g)
    k[5, 0], v[5] = u * (ahead * d ** 0.5 / u.square().sum()), 0
    v[5, 0, 3::32] = 8
    gdn.gdn_kv4_store(x["dims"], k.to(BF).to(DEV), v.to(BF).to(DEV), x["cache"], slot=x["slot"].to(DEV))
    check(x)


def test_scale_is_the_callers():
    x = build(2, 1, 8, 2, 64, 16, [40, 90], seed=7)
    x["dims"].scale = 0.3
    check(x, 0.3)


def test_what_a_query_does_not_see_does_not_reach_it():
    # the last tokens hold NaN and infinities; earlier queries do not see them, later ones do
    x = build(2, 4, 4, 1, 128, 16, [50, 17], seed=8, gate=False)
    clean = call(x)
    k = torch.full((2, 1, 128), float("nan"), dtype=BF, device=DEV)
    last = x["slot"][[49, 66]].to(DEV)
    gdn.gdn_kv4_store(x["dims"], k, k, x["cache"], slot=last)
    got = call(x)
    assert torch.equal(got[:, :3], clean[:, :3])
    assert torch.isnan(got[:, 3]).all()
    v = torch.ones(2, 1, 128, dtype=BF, device=DEV)
    v[0, 0, 40] = float("inf")                 # a group of V alone
    gdn.gdn_kv4_store(x["dims"], torch.zeros_like(v), v, x["cache"], slot=last)
    got = call(x)
    assert torch.equal(got[:, :3], clean[:, :3])
    nan = torch.isnan(got[0, 3])
    assert nan[:, 32:64].all() and not nan[:, :32].any() and not nan[:, 64:].any() and not torch.isnan(got[1]).any()


def test_values_at_the_ends_of_bf16():
    for size in (3.0e38, 2.0 ** -88):
        x = build(1, 1, 8, 1, 64, 16, [100], seed=9, gate=False)
        v = (torch.rand(100, 1, 64, generator=torch.Generator().manual_seed(1)) * 2 - 1) * size
        gdn.gdn_kv4_store(x["dims"], None, v.to(BF).to(DEV), x["cache"], slot=x["slot"].to(DEV))
        check(x)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_of_values_that_differ_by_many_orders(d):
    # tokens' values from 2^-60 to 2^60, small ones first and then in any order; an output is
    # held against the largest magnitudes that reach it
    for order in (False, True):
        x = build(2, 1, 8, 1, d, 32, [700, 333], seed=15, gate=False)
        g = torch.Generator().manual_seed(d)
        e = torch.linspace(-60, 60, 1033)[torch.randperm(1033, generator=g) if order else torch.arange(1033)]
        v = torch.randn(1033, 1, d, generator=g) * torch.exp2(e)[:, None, None]
        gdn.gdn_kv4_store(x["dims"], None, v.to(BF).to(DEV), x["cache"], slot=x["slot"].to(DEV))
        check(x)


def test_groups_that_differ_by_many_orders():
    # a token's groups of channels from 2^-9 to 2^9: each output against its own group's size,
    # except that a weight times a scale below 2^-14 of fp16's top loses bits below 2^-24
    x = build(1, 1, 8, 1, 256, 32, [500], seed=16, gate=False)
    v = torch.randn(500, 1, 8, 32, generator=torch.Generator().manual_seed(3))
    v = (v * torch.exp2(torch.linspace(-9, 9, 8))[:, None]).flatten(-2)
    gdn.gdn_kv4_store(x["dims"], None, v.to(BF).to(DEV), x["cache"], slot=x["slot"].to(DEV))
    check(x)


@pytest.mark.parametrize("S", [1, 3])
def test_rows_of_any_size(S):
    # rows of q of zeros, of subnormal and of huge numbers, with keys that keep the scores ordinary
    x = build(3, S, 8, 1, 128, 32, [100, 65, 40], seed=17, gate=False)
    size = torch.tensor([0.0, 2.0 ** -126, 2.0 ** -130, 2.0 ** -60, 1.0, 2.0 ** -20, 3.0, 2.0 ** 6], device=DEV)
    x["q"] = (x["q"].float() * size[:, None]).to(BF).contiguous()
    check(x)
    for up in (100, -100):                     # (q below 2^108)
        y = build(1, S, 8, 1, 128, 32, [100], seed=18, gate=False)
        y["q"] = (y["q"].float() * 2.0 ** up).to(BF)
        # keys of 2^-88 at the least are held
        k = torch.randn(100, 1, 128, generator=torch.Generator().manual_seed(4)) * 2.0 ** (-86 if up > 0 else 100)
        gdn.gdn_kv4_store(y["dims"], k.to(BF).to(DEV), None, y["cache"], slot=y["slot"].to(DEV))
        y["dims"].scale = 2.0 ** (-17 if up > 0 else -4)
        check(y, y["dims"].scale)


def test_channels_of_a_row_that_differ_by_many_orders():
    # the largest channel meets keys of zero: the scores hang on the small ones
    x = build(1, 1, 8, 1, 128, 32, [300], seed=19, gate=False)
    x["q"][..., 7] = 4096.0
    k = torch.randn(300, 1, 128, generator=torch.Generator().manual_seed(5))
    k[..., :32] = 0
    gdn.gdn_kv4_store(x["dims"], k.to(BF).to(DEV), None, x["cache"], slot=x["slot"].to(DEV))
    check(x)


def test_a_nan_in_the_middle_reaches_every_row_that_sees_it():
    x = build(2, 2, 8, 2, 128, 16, [400, 90], seed=20, gate=False)
    clean = call(x)
    at = x["slot"][[200]].to(DEV)
    bad = torch.ones(1, 2, 128, dtype=BF, device=DEV)
    bad[0, 1, 70] = float("nan")
    gdn.gdn_kv4_store(x["dims"], None, bad, x["cache"], slot=at)     # a group of V of one head
    got = call(x)
    nan = torch.isnan(got)
    assert nan[0, :, 4:, 64:96].all() and not nan[0, :, :4].any() and not nan[0, :, 4:, :64].any()
    assert not nan[0, :, 4:, 96:].any() and torch.equal(got[1], clean[1])
    gdn.gdn_kv4_store(x["dims"], bad, None, x["cache"], slot=at)     # and of K
    got = call(x)
    assert torch.isnan(got[0, :, 4:]).all() and not torch.isnan(got[0, :, :4]).any() and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("d,hq,hk,S", [(256, 32, 2, 4), (256, 16, 2, 8), (128, 40, 8, 2), (64, 64, 1, 2)])
def test_many_rows_over_many_jobs(d, hq, hk, S):
    g = torch.Generator().manual_seed(d)
    check(build(24, S, hq, hk, d, 16, torch.randint(0, 900, (24,), generator=g).tolist(), seed=21))


def test_infinite_scores_follow_the_formula():
    x = build(1, 1, 1, 1, 64, 16, [20], seed=10, gate=False)
    x["q"][0, 0, 0, 3] = float("inf")
    k = torch.ones(20, 1, 64, dtype=BF)
    gdn.gdn_kv4_store(x["dims"], (-k).to(DEV), None, x["cache"], slot=x["slot"].to(DEV))
    assert torch.isnan(call(x)).all()          # all scores -inf
    gdn.gdn_kv4_store(x["dims"], k[:1].to(DEV), None, x["cache"], slot=x["slot"][:1].to(DEV))
    assert torch.isnan(call(x)).all()          # one +inf


def test_bad_lengths_and_pages_are_named():
    x = build(4, 1, 4, 2, 64, 16, [40, 40, 40, 40], seed=11)
    good = call(x)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x["lens"][1] = 1000                        # past the table
    x["lens"][2] = -1
    got = call(x, status=status)
    assert gdn.gdn_read_device_status(status) == gdn.GDN_ERR_DEVICE_BOUNDS
    assert (got[1:3] == 0).all() and torch.equal(got[3], good[3]) and torch.equal(got[0], good[0])
    x["lens"][1:3] = 40
    for bad in (-1, x["cache"].shape[0], 2 ** 31 - 1):
        y = dict(x, table=x["table"].clone())
        y["table"][2, 1] = bad
        status.zero_()
        got = call(y, status=status)
        assert gdn.gdn_read_device_status(status) == gdn.GDN_ERR_DEVICE_BOUNDS
        assert torch.equal(got[[0, 1, 3]], good[[0, 1, 3]])


def test_shared_pages_and_equal_calls():
    x = build(5, 1, 16, 2, 256, 64, [500, 0, 0, 0, 0], seed=12)
    x["table"][1:] = x["table"][0]             # every sequence reads the first one's pages
    x["lens"][1:] = torch.tensor([500, 130, 64, 1], dtype=torch.int32)
    one = call(x)
    assert torch.equal(one, call(x))
    y = dict(x, host=[500], slot=x["slot"])
    for b, n in enumerate([500, 500, 130, 64, 1]):
        z = dict(x, q=x["q"][b:b + 1], gate=x["gate"][b:b + 1], host=[n], slot=x["slot"][:n])
        want, size = reference(z)
        tol = 2 ** -8 * want.abs() + 2 ** -10 * size
        assert ((one[b:b + 1].double() - want).abs() <= tol).all()


def test_captured_step_follows_the_lengths():
    x = build(3, 1, 8, 2, 128, 16, [90, 40, 161], seed=13)
    ws = torch.empty(gdn.gdn_attn_decode_kv4_workspace_bytes(x["dims"], 3, 1), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(x["q"])
    run = lambda: gdn.gdn_attn_decode_kv4(x["dims"], x["q"], x["cache"], x["table"], x["lens"], out, ws)   # noqa: E731
    x["gate"] = None
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lens in ([90, 40, 161], [1, 40, 0], [96, 33, 100]):
        x["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()                         # (96 and 100: two rows hold tokens that were never stored, NaN)
        torch.testing.assert_close(out, call(x), rtol=0, atol=0, equal_nan=True)


def test_two_streams_at_once():
    xs = [build(4, 1, 16, 2, 256, 64, [3000, 10, 500, 1200], seed=20 + i) for i in range(2)]
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(call(xs[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


def test_rows_past_32_bits_of_bytes():
    # one page table entry per end of a cache of 4.8 GB
    dims = gdn.make_attn_dims(h_q=16, h_kv=2, d=256, rot=0)
    pages = 1 << 14
    cache = torch.full((pages, 2, 16, 18 * 256), 255, dtype=torch.uint8, device=DEV)
    x = build(1, 1, 16, 2, 256, 256, [300], seed=14, gate=False)
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=DEV)
    cache[table[0].long()] = x["cache"][x["table"][0].long()]
    got = call(dict(x, cache=cache, table=table))
    assert torch.equal(got, call(x))
