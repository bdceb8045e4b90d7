"""Which experts gdn_moe_step chooses, against logits in 64 bits.

A lane of the router adds n = 4 ceil(hidden / 256) products to each of two
compensated sums (a running sum S and the sum of what its additions dropped),
and six joins follow.  The products are exact in fp32.  With u = 2^-24, each of
the n + 6 additions drops at most u sum |x w|, and their own sum in fp32 loses
at most (n + 6) u of what was dropped: an error below ((n + 6) u)^2 sum |x w|,
half of that on the average over the growing sums.  Two logits are in their
exact order when they are further apart than both errors.  The pairs of experts
here differ by 4 ((hidden / 64 + 6) u)^2 sum |x w| or more, 2^-34 of sum |x w|
at hidden 2048: ordinary fp32 sums (2^-24 and more) decide such a pair by chance.
"""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def route(x, wr, k, renorm=1, sg=None):
    T, H, E = x.shape[0], x.shape[1], wr.shape[0]
    Is = 8 if sg is not None else 0
    dims = gdn.make_moe_dims(hidden=H, inter=8, experts=E, top_k=k, shared_inter=Is, renorm=renorm)
    g = torch.Generator().manual_seed(1)
    r = lambda *s: (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(BF).to(DEV)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    wts = torch.full((T, k), -1.0, device=DEV)
    y = torch.full((T, H), -1.0, device=DEV)
    ws = torch.full((gdn.gdn_moe_step_workspace_bytes(dims, T),), 255, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    gdn.gdn_moe_step(dims, x.to(DEV), wr.to(DEV), r(E, 16, H), r(E, H, 8), y, ws,
                     w_shared_gate_up=r(16, H) if Is else None, w_shared_down=r(H, 8) if Is else None,
                     w_shared_gate=sg.to(DEV) if Is else None, topk_id=ids, topk_w=wts, device_status=st)
    assert gdn.gdn_read_device_status(st) == 0
    return ids.cpu().long(), wts.cpu().double(), y.cpu()


@pytest.mark.parametrize("scale", [1e-18, 1e-4, 1e-2, 1.0, 3e2, 1e4, 1e15])
@pytest.mark.parametrize("T,H", [(1, 64), (8, 2048), (11, 2056), (9, 4096), (5, 8192), (2, 16384)])
def test_near_ties_of_many_terms(T, H, scale):
    g = torch.Generator().manual_seed(H + T)
    E = 32
    x = torch.randn(T, H, generator=g)
    x[:, 1::2] = x[:, ::2]                                   # equal neighbours
    x = x.to(BF)
    w = (torch.randn(E, H, generator=g) * H ** -0.5).to(BF)
    n, size = H // 64, float((x.double().abs() @ w.double().abs().t()).max())
    gap = 4 * ((n + 6) * 2.0 ** -24) ** 2 * size
    # expert 2 i + 1 is expert 2 i with its neighbours exchanged, so that the exact logits
    # are equal, but for one term more, its sign the token's
    swapped = w[::2].view(E // 2, H // 2, 2).flip(-1).reshape(E // 2, H)
    w[1::2] = swapped
    last = H - 2
    x[:, last:] = 0
    term = 2.0 ** torch.randint(0, 3, (E // 2,), generator=g)
    w[::2, last:], w[1::2, last:] = 0, 0
    w[1::2, last] = term.to(BF)
    sign = 1.0 - 2.0 * torch.randint(0, 2, (T,), generator=g)
    x[:, last] = (sign * gap * 1.01).to(BF)                  # (half a step of bf16 is less than 1.01 / 1)
    x[:, last] = torch.where(x[:, last].abs().double() < gap, (x[:, last].double() * 1.01).to(BF), x[:, last])
    assert (x[:, last].double().abs() >= gap).all()
    x = (x.double() * 2.0 ** round(float(torch.log2(torch.tensor(scale))))).to(BF)
    logits = x.double() @ w.double().t()
    # (the 64-bit reference itself is good to 2^-53 H of the sizes, far below the gap)
    order = torch.sort(-logits, dim=-1, stable=True).indices
    ids, _, _ = route(x, w, E)
    assert torch.equal(ids, order)


@pytest.mark.parametrize("scale", [1e-4, 1.0, 20.0])
@pytest.mark.parametrize("H", [2048, 16384])
def test_weights_of_long_rows(H, scale):
    # the rows take several passes through shared memory from hidden 2056 on.  A weight is
    # off by the roundings of two exponentials, a sum of 64 and a division: 2^-20
    g = torch.Generator().manual_seed(H)
    x = (torch.randn(9, H, generator=g) * scale).to(BF)
    w = (torch.randn(64, H, generator=g) * H ** -0.5).to(BF)
    for renorm in (0, 1):
        ids, wts, _ = route(x, w, 6, renorm)
        p = torch.softmax(x.double() @ w.double().t(), -1)
        order = torch.sort(-(x.double() @ w.double().t()), dim=-1, stable=True).indices[:, :6]
        assert torch.equal(ids, order)
        want = p.gather(1, order)
        if renorm:
            want = want / want.sum(-1, keepdim=True)
        assert ((wts - want).abs() <= 2.0 ** -20 * want + 2.0 ** -149).all()


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("H", [64, 2056])
def test_a_router_row_that_is_not_finite_shows(H, renorm):
    g = torch.Generator().manual_seed(7)
    x = torch.randn(5, H, generator=g).to(BF)
    x[:, 11] = torch.tensor([1.0, 2.0, 0.5, 3.0, -1.0]).to(BF)
    w = (torch.randn(40, H, generator=g) * H ** -0.5).to(BF)
    good_ids, good_w, good_y = route(x, w, 4, renorm)
    for value in (NAN, INF, -INF):
        bad = w.clone()
        bad[17, 11] = value                       # logits NaN, or infinite of the token's sign
        ids, wts, y = route(x, bad, 4, renorm)
        for t in range(5):
            logits = x[t].double() @ bad.double().t()
            p = torch.softmax(logits, -1)         # NaN throughout with a NaN or a positive infinity
            assert len(set(ids[t].tolist())) == 4 and (ids[t] >= 0).all() and (ids[t] < 40).all()
            if p.isnan().any():
                assert wts[t].isnan().all() and y[t].isnan().all()
                assert bool((logits == INF).any()) == (17 in ids[t].tolist())
            else:                                 # a weight of zero, the others as they would be
                order = torch.sort(-logits, stable=True).indices[:4]
                assert torch.equal(ids[t], order)
                want = p[order] / (p[order].sum() if renorm else 1.0)
                assert ((wts[t] - want).abs() <= 2.0 ** -20 * want).all() and y[t].isfinite().all()


def test_an_infinite_gate_of_the_shared_expert_opens_or_closes_it():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 64, generator=g).to(BF)
    x[:, 5] = torch.tensor([1.0, -1.0]).to(BF)
    w = (torch.randn(8, 64, generator=g) * 0.1).to(BF)
    sg = torch.zeros(64, dtype=BF)
    sg[5] = INF
    far = sg.clone()
    far[5] = 200.0                                # its sigmoid is 1 or 0 in fp32
    _, _, a = route(x, w, 2, sg=sg)
    _, _, b = route(x, w, 2, sg=far)
    assert torch.equal(a, b)


def test_choosing_a_damaged_expert_among_all():
    # every expert chosen: the NaN one comes last, and the weights are NaN
    g = torch.Generator().manual_seed(9)
    x = torch.randn(3, 64, generator=g).to(BF)
    w = (torch.randn(6, 64, generator=g) * 0.1).to(BF)
    w[2, 0] = NAN
    for renorm in (0, 1):
        ids, wts, y = route(x, w, 6, renorm)
        assert (ids[:, 5] == 2).all() and wts.isnan().all() and y.isnan().all()
