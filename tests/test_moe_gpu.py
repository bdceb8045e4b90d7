"""gdn_moe_step against the layer's definition in 64 bits.

Tolerance.  A gate or up product g = sum x w is summed in fp32 over groups of
partial sums: its error is below 2^-18 sum |x w| (64 steps).  silu has a slope
of at most 1.1, so the activation's error is 1.1 |u| dg + |silu g| du + 2^-16
|a| (a pair of bf16).  The down product passes that on through |w_down| and
adds 2^-18 of its own sum of sizes; a bf16 output adds 2^-8 |y|.
"""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


def inputs(T, H, I, E, Is, seed=0, gate=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda std, *s: (torch.randn(*s, generator=g) * std).to(BF)
    w = dict(x=r(1, T, H), wr=r(H ** -0.5, E, H), gu=r(H ** -0.5, E, 2 * I, H), dn=r(I ** -0.5, E, H, I))
    w.update(sgu=r(H ** -0.5, 2 * Is, H) if Is else None, sdn=r(Is ** -0.5, H, Is) if Is else None,
             sg=r(H ** -0.5, H) if Is and gate else None)
    return w


def expert(x, gu, dn):
    """value, error bound of one expert on rows x (float64)."""
    I = dn.shape[1]
    gu, dn = gu.double(), dn.double()
    p, s = x @ gu.t(), x.abs() @ gu.abs().t()
    g, u, dg, du = p[:, :I], p[:, I:], 2.0 ** -18 * s[:, :I], 2.0 ** -18 * s[:, I:]
    sg = g * torch.sigmoid(g)
    a = sg * u
    da = 1.1 * u.abs() * dg + sg.abs() * du + 2.0 ** -16 * a.abs()
    return a @ dn.t(), da @ dn.abs().t() + 2.0 ** -18 * (a.abs() @ dn.abs().t())


def reference(w, k, renorm):
    x = w["x"].double()
    T = x.shape[0]
    logits = x @ w["wr"].double().t()
    ids = torch.sort(-logits, dim=-1, stable=True).indices[:, :k]
    p = torch.softmax(logits, -1).gather(1, ids)
    if renorm:
        p = p / p.sum(-1, keepdim=True)
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        for j in range(k):
            v, e = expert(x[t:t + 1], w["gu"][ids[t, j]], w["dn"][ids[t, j]])
            y[t] += p[t, j] * v[0]
            tol[t] += p[t, j] * (e[0] + 2.0 ** -20 * v[0].abs())
    if w["sgu"] is not None:
        v, e = expert(x, w["sgu"], w["sdn"])
        f = torch.sigmoid(x @ w["sg"].double()) if w["sg"] is not None else torch.ones(T, dtype=torch.float64)
        y += f[:, None] * v
        tol += f[:, None] * (e + 2.0 ** -18 * v.abs())
    return y, tol, ids, p


def call(dims, w, dtype=F32, stream=None):
    T = w["x"].shape[0]
    d = {k: (v.to(DEV) if v is not None else None) for k, v in w.items()}
    y = torch.full((T, dims.hidden), float("nan"), dtype=dtype, device=DEV)
    ids = torch.full((T, dims.top_k), -1, dtype=torch.int32, device=DEV)
    wts = torch.full((T, dims.top_k), -1.0, device=DEV)
    ws = torch.full((gdn.gdn_moe_step_workspace_bytes(dims, T),), 255, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    gdn.gdn_moe_step(dims, d["x"], d["wr"], d["gu"], d["dn"], y, ws, w_shared_gate_up=d["sgu"],
                     w_shared_down=d["sdn"], w_shared_gate=d["sg"], topk_id=ids, topk_w=wts, device_status=st)
    assert gdn.gdn_read_device_status(st) == 0
    return y, ids, wts


def check(w, I, k, renorm, dtype):
    T, H = w["x"].shape
    E = w["wr"].shape[0]
    Is = 0 if w["sgu"] is None else w["sdn"].shape[1]
    dims = gdn.make_moe_dims(hidden=H, inter=I, experts=E, top_k=k, shared_inter=Is, renorm=int(renorm))
    y, ids, wts = call(dims, w, dtype)
    ref, tol, rid, rw = reference(w, k, renorm)
    assert torch.equal(ids.cpu().long(), rid)
    assert ((wts.cpu().double() - rw).abs() <= 2.0 ** -20 * rw + 2.0 ** -149).all()   # a subnormal step
    if dtype == BF:
        tol = tol + 2.0 ** -8 * ref.abs()
    got = y.double().cpu()
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() - tol
    assert (bad <= 0).all(), float(bad.max())
    return y


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,H,I,E,k,Is,renorm", [
    (1, 8, 8, 1, 1, 0, True), (1, 64, 16, 4, 2, 8, True), (2, 520, 24, 3, 3, 0, False), (3, 1032, 136, 16, 4, 72, True),
    (1, 2048, 512, 32, 8, 512, True), (7, 256, 1032, 8, 2, 0, False), (8, 128, 64, 64, 6, 64, True),
    (9, 1000, 40, 5, 5, 24, False), (17, 512, 128, 24, 3, 0, True), (33, 264, 48, 7, 2, 40, True),
    (64, 512, 256, 16, 4, 128, False), (64, 136, 8, 200, 10, 0, True), (5, 64, 32, 1024, 32, 0, True)])
def test_matches_the_definition(T, H, I, E, k, Is, renorm, dtype):
    check(inputs(T, H, I, E, Is, seed=T + H), I, k, renorm, dtype)


def test_all_tokens_to_one_expert_and_shared_without_gate():
    w = inputs(64, 256, 64, 12, 32, gate=False)
    w["x"][:] = w["x"][0]                       # every token takes the same experts
    check(w, 64, 3, True, F32)
    y = check(w, 64, 1, True, F32)
    assert (y == y[0]).all()


def test_ties_go_to_the_lowest_index():
    w = inputs(6, 128, 16, 40, 0)
    w["wr"][1::2] = w["wr"][::2]                # pairs of equal logits
    check(w, 16, 5, True, F32)
    w["wr"][:] = w["wr"][0]                     # all alike
    y, ids, wts = call(gdn.make_moe_dims(hidden=128, inter=16, experts=40, top_k=7), w)
    assert (ids.cpu() == torch.arange(7)).all() and torch.allclose(wts.cpu(), torch.full((6, 7), 1 / 7))


def test_near_ties_follow_the_exact_logits():
    # logits that differ by less than fp32 holds at their size: 2^-26 against 8
    w = inputs(2, 64, 16, 6, 0)
    w["x"][:] = 1.0
    w["wr"][:] = 0.0
    w["wr"][:, 0] = 8.0
    w["wr"][4, 1] = 2.0 ** -26
    w["wr"][2, 2] = 2.0 ** -27
    _, ids, _ = call(gdn.make_moe_dims(hidden=64, inter=16, experts=6, top_k=3), w)
    assert ids.cpu().tolist() == [[4, 2, 0]] * 2


def test_large_logits_and_small_probabilities():
    w = inputs(4, 256, 32, 10, 0)
    w["wr"] = (w["wr"].float() * 60).to(BF)     # logits of a hundred: most probabilities vanish
    check(w, 32, 3, True, F32)
    # a chosen weight that underflows without renorm is zero, not NaN
    y, _, wts = call(gdn.make_moe_dims(hidden=256, inter=32, experts=10, top_k=10, renorm=0), w)
    assert torch.isfinite(y).all() and torch.isfinite(wts).all()


def test_a_token_does_not_depend_on_the_others():
    w = inputs(64, 512, 136, 32, 64, seed=3)
    dims = gdn.make_moe_dims(hidden=512, inter=136, experts=32, top_k=4, shared_inter=64)
    y, ids, wts = call(dims, w)
    for pick in ([5], [9, 5], list(range(0, 23)), list(range(40, 64))):
        a, b, c = call(dims, dict(w, x=w["x"][pick]))
        assert torch.equal(a, y[pick]) and torch.equal(b, ids[pick]) and torch.equal(c, wts[pick])


def test_unused_experts_are_not_read_into_the_sum():
    w = inputs(3, 128, 32, 20, 0)
    dims = gdn.make_moe_dims(hidden=128, inter=32, experts=20, top_k=2)
    y, ids, _ = call(dims, w)
    used = set(ids.flatten().tolist())
    for e in range(20):
        if e not in used:
            w["gu"][e] = float("nan")
            w["dn"][e] = float("inf")
    assert torch.equal(call(dims, w)[0], y)


def test_a_bad_token_stays_alone():
    w = inputs(10, 264, 40, 6, 16)
    dims = gdn.make_moe_dims(hidden=264, inter=40, experts=6, top_k=2, shared_inter=16)
    y, ids, _ = call(dims, w)
    w["x"][4, 7] = float("nan")
    z, jds, _ = call(dims, w)
    keep = [t for t in range(10) if t != 4]
    assert torch.equal(z[keep], y[keep]) and torch.equal(jds[keep], ids[keep])
    assert ((jds >= 0) & (jds < 6)).all() and len(set(jds[4].tolist())) == 2


def test_streams_graphs_and_repeated_calls():
    w = inputs(5, 512, 64, 16, 32)
    dims = gdn.make_moe_dims(hidden=512, inter=64, experts=16, top_k=3, shared_inter=32)
    y, ids, wts = call(dims, w)
    d = {k: v.to(DEV) for k, v in w.items()}
    ws = torch.empty(gdn.gdn_moe_step_workspace_bytes(dims, 5), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(y)

    def step():
        gdn.gdn_moe_step(dims, d["x"], d["wr"], d["gu"], d["dn"], out, ws, w_shared_gate_up=d["sgu"],
                         w_shared_down=d["sdn"], w_shared_gate=d["sg"])

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(20):
            step()
    s.synchronize()
    assert torch.equal(out, y)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
        step()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
