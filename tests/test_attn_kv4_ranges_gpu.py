"""gdn_attn_decode_kv4 where V's magnitudes lie many binary orders apart: between tokens that a
row sees and does not see, weighs and hardly weighs, and between groups of channels.

Tolerance: test_attn_kv4_gpu's, and for each token that the row sees, of weight p and with
magnitudes up to M in the value's group, min(p, 2^-22 P) M, P the row's largest weight.  A
weight times a scale is an fp16 number, of scales within 10 binary orders below the power
of two that they are taken relative to; the largest weight so far lies above 2^7 there.  Below
fp16's normal numbers a rounding is off by at most 2^-25, which is 2^-32 P of that power of two,
2^-22 P of the least scale times 8 codes, and no more than the number itself."""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
from test_attn_kv4_gpu import BF, DEV, build, call, values
from test_attn_kv4_sums_gpu import many

pytestmark = pytest.mark.gpu


def errors(x, S, lens):
    """Errors of every output in units of the tolerance ([B, S, h_kv, G, d])."""
    k_all, v_all = values(x)
    B, _, hq, d = x["q"].shape
    hk = x["dims"].h_kv
    q = x["q"].double().unflatten(2, (hk, hq // hk))
    got = call(x).double().unflatten(2, (hk, hq // hk))
    most_all = v_all.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
    out, at = torch.zeros_like(got), 0
    for b, n in enumerate(lens):
        for i in range(S):
            m = n - S + 1 + i
            k, v, most = k_all[at:at + m], v_all[at:at + m], most_all[at:at + m]
            p = torch.softmax(torch.einsum("nhd,hgd->hgn", k, q[b, i]) * d ** -0.5, -1)
            want = torch.einsum("hgn,nhd->hgd", p, v)
            size = torch.einsum("hgn,nhd->hgd", p, v.abs() + 2 ** -6 * most)
            lost = torch.einsum("hgn,nhd->hgd", torch.minimum(p, 2 ** -22 * p.amax(-1, keepdim=True)), most)
            tol = 2 ** -8 * want.abs() + 2 ** -10 * size + lost + 1e-40
            out[b, i] = ((got[b, i] - want).abs() / tol).nan_to_num(nan=float("inf"))
        at += n
    return out


def stored(B, S, G, d, lens, k, v, seed):
    x = build(B, S, 2 * G, 2, d, 16, lens, seed=seed, gate=False)
    gdn.gdn_kv4_store(x["dims"], None if k is None else k.to(BF).to(DEV), v.to(BF).to(DEV), x["cache"],
                      slot=x["slot"].to(DEV))
    return x


SHAPES = [(64, 1, 4), (64, 2, 8), (128, 1, 8), (128, 2, 5), (256, 1, 8), (256, 2, 4), (256, 4, 4)]


@pytest.mark.parametrize("d,G,S", [(64, 1, 4), (64, 4, 4), (128, 2, 2), (128, 4, 4), (256, 2, 3), (256, 4, 3)])
@pytest.mark.parametrize("up", [12, 40, 120])
def test_values_that_a_query_does_not_see_do_not_reach_it(d, G, S, up):
    lens = [50, 17, 300]
    g = torch.Generator().manual_seed(d + up)
    v = torch.randn(sum(lens), 2, d, generator=g)
    x = stored(3, S, G, d, lens, None, v, seed=30)
    assert errors(x, S, lens).max() <= 1
    last = [sum(lens[:b + 1]) - 1 for b in range(3)]
    v[last] *= 2.0 ** up
    x = stored(3, S, G, d, lens, None, v, seed=30)
    worst = errors(x, S, lens)
    assert worst[:, :S - 1].max() <= 1, worst[:, :S - 1].max()
    assert worst.max() <= 1, worst.max()


@pytest.mark.parametrize("d,S,G", SHAPES)
@pytest.mark.parametrize("up,down", [(20, 40), (40, 80), (100, 180)])
def test_large_values_with_hardly_any_weight_leave_the_others(d, S, G, up, down):
    # one token's score lies `down` binary orders below the others', its values 2^up above
    n = 150
    g = torch.Generator().manual_seed(d + up)
    u = torch.randn(d, generator=g)
    k, v = 0.1 * torch.randn(n, 2, d, generator=g), torch.randn(n, 2, d, generator=g)
    for at in (3, 70):                         # in the first stage and in a later one
        k[at] = -u * (down * 0.6931 * d ** 0.5 / u.square().sum())
        v[at] *= 2.0 ** up
    x = stored(1, S, G, d, [n], k, v, seed=31)
    x["q"] = (u + 0.05 * torch.randn(1, S, 2 * G, d, generator=g)).to(BF).to(DEV)
    worst = errors(x, S, [n]).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("d,S,G", SHAPES)
@pytest.mark.parametrize("apart", [12, 24, 30, 60, 150])
def test_groups_far_apart_keep_their_own_precision(d, S, G, apart):
    n = 333
    R = d // 32
    v = torch.randn(n, 2, R, 32, generator=torch.Generator().manual_seed(d))
    e = torch.linspace(-apart / 2, apart / 2, R)
    v = (v * torch.exp2(e)[:, None]).flatten(-2)
    worst = errors(stored(1, S, G, d, [n], None, v, seed=32), S, [n]).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("d,S,G", SHAPES)
@pytest.mark.parametrize("low,high", [(-89, -68), (-86, -76), (105, 125), (113, 126)])
def test_groups_apart_at_the_ends_of_the_range(d, S, G, low, high):
    n = 150
    R = d // 32
    v = torch.rand(n, 2, R, 32, generator=torch.Generator().manual_seed(d)) + 0.5
    e = torch.linspace(low, high, R)
    v = (v * torch.exp2(e)[:, None]).flatten(-2)
    worst = errors(stored(1, S, G, d, [n], None, v, seed=36), S, [n]).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("d,S,G", SHAPES)
def test_every_token_and_group_of_a_size_of_its_own(d, S, G):
    lens = [333, 90, 5]
    n, R = sum(lens), d // 32
    g = torch.Generator().manual_seed(d + G)
    e = torch.rand(n, 2, R, 1, generator=g) * 200 - 85     # (held from 2^-90 on)
    v = (torch.randn(n, 2, R, 32, generator=g) * torch.exp2(e)).flatten(-2)
    v[torch.rand(n, generator=g) < 0.1] = 0
    worst = errors(stored(3, S, G, d, lens, None, v, seed=33), S, lens).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("d,S,G", [(64, 1, 4), (128, 4, 4), (256, 1, 8), (256, 4, 4)])
def test_sizes_that_go_up_and_down_within_a_share(d, S, G):
    # shares of whole jobs, the same tokens for all of them
    n = 260
    g = torch.Generator().manual_seed(d)
    e = 30 * torch.randint(-2, 4, (n // 20, 1), generator=g).repeat_interleave(20, 0).float()
    k, v = torch.randn(n, 8, d, generator=g), torch.randn(n, 8, d, generator=g) * torch.exp2(e)[..., None]
    x = many(S, G, d, n, k, v, seed=34)
    some = [0, 1, 100, 255, 400, 511]
    whole = call(x)
    y = dict(x, q=x["q"][some], table=x["table"][some], lens=x["lens"][some])
    worst = errors_of(whole[some], y, S, n)
    assert worst <= 1, worst


def errors_of(got, x, S, n):
    k, v = values(x)
    hk = x["dims"].h_kv
    q, got = (t.double().unflatten(2, (hk, -1)) for t in (x["q"], got))
    d = q.shape[-1]
    most = v.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
    worst = 0.0
    for i in range(S):
        m = n - S + 1 + i
        p = torch.softmax(torch.einsum("nhd,bhgd->bhgn", k[:m], q[:, i]) * d ** -0.5, -1)
        want = torch.einsum("bhgn,nhd->bhgd", p, v[:m])
        size = torch.einsum("bhgn,nhd->bhgd", p, v[:m].abs() + 2 ** -6 * most[:m])
        lost = torch.einsum("bhgn,nhd->bhgd", torch.minimum(p, 2 ** -22 * p.amax(-1, keepdim=True)), most[:m])
        tol = 2 ** -8 * want.abs() + 2 ** -10 * size + lost + 1e-36
        worst = max(worst, ((got[:, i] - want).abs() / tol).nan_to_num(nan=float("inf")).max().item())
    return worst


@pytest.mark.parametrize("d,S,G", SHAPES)
def test_a_nan_next_to_values_of_many_sizes(d, S, G):
    # a NaN group of V stays in its group, whatever sizes the others have
    n = 200
    g = torch.Generator().manual_seed(d)
    v = torch.randn(n, 2, d // 32, 32, generator=g) * torch.exp2(40 * torch.rand(n, 2, d // 32, 1, generator=g) - 20)
    x = stored(1, S, G, d, [n], None, v.flatten(-2), seed=35)
    clean = call(x)
    assert errors(x, S, [n]).max() <= 1
    bad = v.flatten(-2)[100:101].clone()
    bad[0, 1, 5] = float("nan")                # group 0 of head 1
    gdn.gdn_kv4_store(x["dims"], None, bad.to(BF).to(DEV), x["cache"], slot=x["slot"][100:101].to(DEV))
    got = call(x)
    nan = torch.isnan(got)
    assert nan[:, :, G:, :32].all() and not nan[:, :, :G].any() and not nan[:, :, G:, 32:].any()
    assert torch.equal(got[:, :, :G], clean[:, :, :G])
    assert errors(x, S, [n])[:, :, 1, :, 32:].max() <= 1


def sizes(n, d, seed, span=60):
    """Values of n tokens, groups of a token up to 2^span apart."""
    g = torch.Generator().manual_seed(seed)
    e = span * torch.rand(n, 2, d // 32, 1, generator=g) - span / 2
    return (torch.randn(n, 2, d // 32, 32, generator=g) * torch.exp2(e)).flatten(-2)


@pytest.mark.parametrize("d,S,G", [s for s in SHAPES if s[1] > 1])
def test_what_is_not_seen_next_to_values_of_many_sizes(d, S, G):
    lens = [100, 64, 37]
    v = sizes(sum(lens), d, 37)
    x = stored(3, S, G, d, lens, None, v, seed=37)
    clean = call(x)
    last = x["slot"][[99, 163, 200]].to(DEV)
    for bad in (float("nan"), 3e38):
        rows = torch.full((3, 2, d), bad, dtype=BF, device=DEV)
        gdn.gdn_kv4_store(x["dims"], rows, rows, x["cache"], slot=last)
        got = call(x)
        if bad == bad:                         # (other passes, other roundings: held to the formula)
            assert errors(x, S, lens)[:, :S - 1].max() <= 1
        else:
            assert torch.equal(got[:, :S - 1], clean[:, :S - 1]) and torch.isnan(got[:, S - 1]).all()


@pytest.mark.parametrize("d,S,G", SHAPES)
def test_long_sequences_of_many_sizes_in_many_shares(d, S, G):
    lens = [9001, 5000]
    v = sizes(sum(lens), d, 38)
    worst = errors(stored(2, S, G, d, lens, None, v, seed=38), S, lens).max()
    assert worst <= 1, worst


@pytest.mark.parametrize("d,S,G", [(64, 1, 4), (128, 4, 4), (256, 1, 8)])
def test_equal_and_captured_calls_on_values_of_many_sizes(d, S, G):
    lens = [700, 33, 0, 260]
    x = stored(4, S, G, d, lens, None, sizes(sum(lens), d, 39), seed=39)
    want = call(x)
    ws = torch.full((gdn.gdn_attn_decode_kv4_workspace_bytes(x["dims"], 4, S),), 255, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    run = lambda: gdn.gdn_attn_decode_kv4(x["dims"], x["q"], x["cache"], x["table"], x["lens"], out, ws)   # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        assert torch.equal(out, want)


def test_scores_that_grow_over_values_of_many_sizes():
    # references move between parts of the sums that stand in memory
    n = 700
    for d, S, G in SHAPES:
        g = torch.Generator().manual_seed(d)
        k = torch.randn(n, 2, d, generator=g) * (0.02 * torch.arange(n)[:, None, None])
        worst = errors(stored(1, S, G, d, [n], k, sizes(n, d, 40), seed=40), S, [n]).max()
        assert worst <= 1, (d, S, G, worst)
