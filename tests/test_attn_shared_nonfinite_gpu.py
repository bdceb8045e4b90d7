"""Infinities and NaN in gdn_attn_decode_shared: they reach every row whose
formula holds them and no other.

Finite results: the tolerance of the finite tests, (2^-8 + 2^-11) A + 2^-8 |o|
with A = sum p |v| (a weight rounded to bf16, fp32 scores and exponentials, one
rounding of the result).  Rows that hold nothing of what was changed keep
their bits.
"""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
from test_attn_shared_gpu import BF, build, call, reference

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def check(dims, x):
    """NaN and infinities where the definition has them, the rest within tolerance."""
    out, st = call(dims, x)
    assert st == 0
    ref, size = reference(x, dims.h_kv, dims.d ** -0.5)
    got = out.double().cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isinf(), ref.isinf()) and (got[ref.isinf()] == ref[ref.isinf()]).all()
    fin = ref.isfinite()
    tol = (2.0 ** -8 + 2.0 ** -11) * size + 2.0 ** -8 * ref.abs()
    assert ((got - ref).abs() <= tol)[fin].all()
    return out


def put_own(x, b, key, k=None, v=None, dims=slice(None)):
    """Key `key` of sequence b's tail, in the cache and in the definition's copy."""
    page = x["kc"].shape[1]
    at = (int(x["tp"][b, key // page]), key % page)
    for cache, ref, val in ((x["kc"], x["seqs"][b][0], k), (x["vc"], x["seqs"][b][1], v)):
        if val is not None:
            cache[at][..., dims] = val
            ref[key][..., dims] = val


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("S,prefix,tails", [(1, 0, [5, 64, 200]), (1, 300, [0, 3, 129]), (2, 2600, [7, 31, 260])])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_query_that_is_not_finite_gives_nan_in_its_row_alone(d, S, prefix, tails, value):
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=d, rot=0)
    x = build(3, S, 4, 2, d, 16, prefix, tails, seed=d)
    good = check(dims, x)
    x["q"][1, S - 1, 2, 7] = value
    out = check(dims, x)
    assert out[1, S - 1, 2].isnan().all()
    keep = torch.ones(3, S, 4, dtype=torch.bool)
    keep[1, S - 1, 2] = False
    assert torch.equal(out[keep], good[keep])


def test_keys_that_are_not_finite_reach_the_rows_that_see_them():
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=128, rot=0)
    x = build(4, 1, 4, 2, 128, 16, 500, [20, 128, 0, 300], seed=2)
    good = check(dims, x)
    for b in (0, 1, 3):              # a whole tail of NaN keys: that sequence, no other
        y = dict(x, kc=x["kc"].clone(), seqs=[(k.clone(), v.clone()) for k, v in x["seqs"]])
        for j in range(x["tails"][b]):
            put_own(y, b, j, k=NAN)
        out = check(dims, y)
        assert out[b].isnan().all()
        rest = [i for i in range(4) if i != b]
        assert torch.equal(out[rest], good[rest])
    # one key of the prefix, one key head: that head's rows
    y = dict(x, kc=x["kc"].clone(), pre=(x["pre"][0].clone(), x["pre"][1]))
    y["kc"][int(x["pp"][20]), 3, 1, 9] = NAN
    y["pre"][0][20 * 16 + 3, 1, 9] = NAN
    out = check(dims, y)
    assert out[:, :, 2:].isnan().all() and torch.equal(out[:, :, :2], good[:, :, :2])


# ---- what a query does not see ----
# With several tokens a sequence, a tail's last tokens are hidden from its earlier
# queries, whatever they hold.

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("S,page,prefix,tails", [
    (4, 16, 0, [4, 9, 16, 2]),                    # from the first token on, and a tail shorter than its queries
    (4, 16, 70, [130, 131, 128, 3]),              # the hidden tokens across two tiles
    (8, 64, 200, [64, 135, 129, 8]), (2, 32, 0, [1, 33, 128, 257]), (3, 128, 1000, [700, 2, 0, 514])])
@pytest.mark.parametrize("bad", ["nan value", "inf value", "both infinities", "nan key", "all of it"])
def test_hidden_tokens_do_not_reach_earlier_queries(d, S, page, prefix, tails, bad):
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=d, rot=0)
    x = build(4, S, 4, 2, d, page, prefix, tails, seed=S + d)
    good = check(dims, x)
    some = slice(d // 2 - 3, d // 2 + 5)          # dimensions of both halves
    for b, n in enumerate(tails):
        if b == 3 or n == 0:
            continue                              # the last sequence stays as it was
        if bad == "nan value":
            put_own(x, b, n - 1, v=NAN, dims=some)
        elif bad == "inf value":
            put_own(x, b, n - 1, v=-INF, dims=some)
        elif bad == "both infinities":            # a row that sees both has a NaN
            put_own(x, b, n - 1, v=INF, dims=some)
            if n > 1:
                put_own(x, b, n - 2, v=-INF, dims=slice(0, d // 2))
        elif bad == "nan key":
            put_own(x, b, n - 1, k=NAN, dims=some)
        else:
            for j in range(max(0, n - S + 1), n):
                put_own(x, b, j, k=NAN, v=NAN)
    out = check(dims, x)
    assert torch.equal(out[3], good[3])
    if bad != "both infinities" or S > 2:         # (of two, every query sees the last token but one)
        assert torch.equal(out[:, 0], good[:, 0])


def test_values_that_every_query_sees_reach_every_query():
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=128, rot=0)
    x = build(2, 3, 4, 2, 128, 16, 90, [40, 50], seed=1)
    put_own(x, 0, 37, v=INF, dims=slice(5, 6))    # the last token that all three see
    put_own(x, 1, 0, v=NAN, dims=slice(70, 80))
    x["vc"][int(x["pp"][5]), 9, 0, 33] = -INF
    x["pre"][1][5 * 16 + 9, 0, 33] = -INF
    out = check(dims, x)
    assert (out[0, :, :, 5] == INF).all() and out[1, :, :, 70:80].isnan().all() and (out[:, :, :2, 33] == -INF).all()
