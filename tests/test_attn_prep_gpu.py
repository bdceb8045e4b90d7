"""gdn_attn_prep against the norm, the rotation and the scatter in 64 bits.

Tolerance: the result is one bf16 rounding (half a step, 2^-8 relative) of an
fp32 chain of about 16 roundings over values no larger than the row's norm
allows; the angle, kept to 2^-24 of a turn, moves a pair by 2 pi 2^-25 of its
length.  Together 2^-8 |ref| + 2^-19 max|row|.
"""
import math

import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def reference(x, w, inv_freq, axis, pos, rot, pairs, eps):
    """[T, H, d] -> float64 [T, H, d] (CPU)."""
    x = x.double().cpu()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double().cpu()
    y, nf = x.clone(), rot // 2
    for i in range(nf):
        phi = pos[axis[i]].double().cpu() * float(inv_freq[i])
        c, s = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + nf)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def close(got, ref):
    got = got.double().cpu()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -19 * ref.abs().amax(-1, keepdim=True)
    bad = (got - ref).abs() - tol
    assert torch.isfinite(got).all() and (bad <= 0).all(), float(bad.max())


def inputs(T, hq, hk, d, rot, axes, seed, far=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    pos = torch.randint(0, 4096, (axes, T), generator=g) + far
    return dict(q=r(T, hq, d).to(BF).to(DEV), k=r(T, hk, d).to(BF).to(DEV), v=r(T, hk, d).to(BF).to(DEV),
                qw=(1 + 0.3 * r(d)).to(DEV), kw=(1 + 0.3 * r(d)).to(DEV),
                inv=torch.tensor([1e6 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64).to(DEV),
                axis=torch.randint(0, axes, (rot // 2,), generator=g).int().to(DEV),
                pos=pos.int().to(DEV), slot=torch.randperm(T + 5, generator=g)[:T].int().to(DEV))


def call(dims, x, rows, **kw):
    T, hk, d = x["q"].shape[0], dims.h_kv, dims.d
    kc = torch.full((rows, hk, d), 7.0, dtype=BF, device=DEV)
    vc = torch.full((rows, hk, d), 7.0, dtype=BF, device=DEV)
    qo = torch.full((T, dims.h_q, d), float("nan"), dtype=BF, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    gdn.gdn_attn_prep(dims, x["q"], x["k"], x["v"], x["qw"], x["kw"], x["inv"], x["axis"], x["pos"], qo, kc, vc,
                      slot=x["slot"], device_status=st, **kw)
    return qo, kc, vc, gdn.gdn_read_device_status(st)


@pytest.mark.parametrize("d,hq,hk,rot,axes,pairs,T", [
    (256, 16, 2, 64, 1, 0, 1), (256, 16, 2, 256, 3, 0, 7), (256, 3, 1, 64, 2, 1, 130), (128, 32, 8, 128, 3, 0, 33),
    (128, 5, 5, 32, 1, 1, 2), (128, 6, 2, 16, 1, 0, 4099), (64, 9, 3, 64, 4, 0, 5), (64, 1, 1, 16, 1, 1, 1),
    (64, 7, 1, 32, 1, 0, 600), (128, 4, 2, 0, 1, 0, 9)])
def test_matches_the_definition(d, hq, hk, rot, axes, pairs, T):
    dims = gdn.make_attn_dims(h_q=hq, h_kv=hk, d=d, rot=rot, n_axes=axes, rope_pairs=pairs, norm_eps=1e-6)
    x = inputs(T, hq, hk, d, max(rot, 2), axes, T + d)
    if rot == 0:
        x["inv"] = x["axis"] = x["pos"] = None
    qo, kc, vc, st = call(dims, x, T + 5)
    assert st == 0
    args = (x["inv"], [0] * rot if axes == 1 else x["axis"].tolist(), x["pos"], rot, pairs, 1e-6) if rot else \
        (None, None, None, 0, pairs, 1e-6)
    close(qo, reference(x["q"], x["qw"], *args))
    rows = x["slot"].long()
    close(kc[rows], reference(x["k"], x["kw"], *args))
    assert torch.equal(vc[rows], x["v"])
    rest = torch.ones(T + 5, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert (kc[rest] == 7).all() and (vc[rest] == 7).all()


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 5000, -3000])
def test_far_positions_lose_nothing(far):
    dims = gdn.make_attn_dims(h_q=2, h_kv=1, d=128, rot=128)
    x = inputs(9, 2, 1, 128, 128, 1, 5)
    x["pos"] = (torch.arange(9) * 11 + far).int()[None].to(DEV)
    qo, _, _, st = call(dims, x, 14)
    # a radian count of 2^31 holds 2^-22 in 64 bits: the reference itself is good to that
    ref = reference(x["q"], x["qw"], x["inv"], [0] * 64, x["pos"], 128, 0, 1e-6)
    assert st == 0
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -19 + 2.0 ** -20) * ref.abs().amax(-1, keepdim=True)
    assert ((qo.double().cpu() - ref).abs() <= tol).all()


def test_strided_views_in_place_and_left_out_parts():
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=64, rot=32)
    x = inputs(21, 4, 2, 64, 32, 1, 3)
    want_q, want_k, want_v, _ = call(dims, x, 26)
    # q inside a [T, h, 2 d] projection with the gate beside it, k and v inside one array
    wide = torch.full((21, 4, 128), float("nan"), dtype=BF, device=DEV)
    wide[..., :64] = x["q"]
    kv = torch.stack([x["k"], x["v"]], 1).contiguous()
    y = dict(x, q=wide[..., :64], k=kv[:, 0], v=kv[:, 1])
    for a, b in zip(call(dims, y, 26)[:3], (want_q, want_k, want_v)):
        assert torch.equal(a, b)
    # in place
    q = x["q"].clone()
    gdn.gdn_attn_prep(dims, q, None, None, x["qw"], None, x["inv"], None, x["pos"], q, None, None)
    assert torch.equal(q, want_q)
    # k and v alone, to rows 0 .. T-1
    kc = torch.zeros(21, 2, 64, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    gdn.gdn_attn_prep(dims, None, x["k"], x["v"], None, x["kw"], x["inv"], None, x["pos"], None, kc, vc)
    assert torch.equal(kc, want_k[x["slot"].long()]) and torch.equal(vc, x["v"])
    # no norm
    gdn.gdn_attn_prep(dims, x["q"], None, None, None, None, x["inv"], None, x["pos"], q, None, None)
    close(q, reference(x["q"], None, x["inv"], [0] * 16, x["pos"], 32, 0, 1e-6))


def test_slots_and_axes_out_of_range():
    dims = gdn.make_attn_dims(h_q=2, h_kv=2, d=64, rot=32, n_axes=2)
    x = inputs(6, 2, 2, 64, 32, 2, 8)
    x["slot"] = torch.tensor([0, -1, 2, -7, 4, 5], dtype=torch.int32, device=DEV)
    _, kc, vc, st = call(dims, x, 6)
    assert st == 0                     # negative: a token that is not stored
    assert (kc[[1, 3]] == 7).all() and (vc[[1, 3]] == 7).all() and torch.equal(vc[[0, 2, 4, 5]], x["v"][[0, 2, 4, 5]])
    x["slot"][4] = 6
    _, kc, vc, st = call(dims, x, 6)
    assert st == gdn.GDN_ERR_DEVICE_BOUNDS and (kc[[1, 3, 4]] == 7).all()
    x["slot"][4] = 4
    x["axis"][3] = 2
    qo, _, _, st = call(dims, x, 6)
    assert st == gdn.GDN_ERR_DEVICE_BOUNDS
    ax = x["axis"].tolist()
    ax[3] = 0
    close(qo, reference(x["q"], x["qw"], x["inv"], ax, x["pos"], 32, 0, 1e-6))


def test_zero_rows_and_infinities_stay_in_their_rows():
    dims = gdn.make_attn_dims(h_q=3, h_kv=1, d=128, rot=64)
    x = inputs(4, 3, 1, 128, 64, 1, 9)
    good = call(dims, x, 9)[0]
    x["q"][1, 0] = 0
    x["q"][2, 1, 5] = float("inf")
    qo = call(dims, x, 9)[0]
    assert (qo[1, 0] == 0).all() and not torch.isfinite(qo[2, 1]).all()
    keep = torch.ones(4, 3, dtype=torch.bool)
    keep[1, 0] = keep[2, 1] = False
    assert torch.equal(qo[keep.to(DEV)], good[keep.to(DEV)])


def test_other_streams_and_graphs():
    dims = gdn.make_attn_dims(h_q=4, h_kv=2, d=128, rot=64)
    x = inputs(50, 4, 2, 128, 64, 1, 4)
    want = call(dims, x, 55)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(dims, x, 55)[0]
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    kc = torch.zeros(55, 2, 128, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_attn_prep(dims, x["q"], x["k"], x["v"], x["qw"], x["kw"], x["inv"], None, x["pos"], out, kc, vc,
                          slot=x["slot"])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_norm_is_held_in_32_bits():
    # rows whose squares leave bf16 and fp16 behind, and whose small terms a 16-bit sum would drop
    dims = gdn.make_attn_dims(h_q=1, h_kv=1, d=256, rot=0)
    q = torch.full((2, 1, 256), 1e-2, dtype=BF, device=DEV)
    q[0, 0, 0] = 1e15
    q[1] *= 1e-15
    x = dict(q=q, k=q, v=q, qw=torch.ones(256, device=DEV), kw=torch.ones(256, device=DEV), inv=None, axis=None,
             pos=None, slot=None)
    qo = call(dims, x, 2)[0]
    ref = reference(q, torch.ones(256), None, None, None, 0, 0, 1e-6)
    assert math.isclose(float(qo[0, 0, 0]), 16.0, rel_tol=2 ** -8)
    close(qo, ref)
