"""gdn_kv4_store and gdn_kv4_load against the format's definition, bit for bit: a code is
the nearest multiple of an exact scale, so there is nothing to be off by.  The loaded
values are a code times its scale: 3 and 8 significant bits, exact in fp32 and rounded
once to bf16."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
import kv4_util as kv4

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


def rows(T, h, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, h, d, generator=g) * scale).to(BF)


def special(T, h, d, seed):
    """Rows with what a group can hold: ties, both signs of the extreme, zeros, the
    smallest and the largest numbers, infinities and NaN."""
    x = rows(T, h, d, seed)
    flat = x.view(-1, 32)
    kinds = [torch.zeros(32), torch.full((32,), -0.0), torch.linspace(-8, 7.5, 32), -torch.linspace(-8, 7.5, 32),
             torch.tensor([1.0, -1.0] * 16), torch.full((32,), 3.3895e38), torch.full((32,), -3.3895e38),
             torch.cat([torch.tensor([3.0e38]), torch.full((31,), 1e-30)]), torch.full((32,), 2.0 ** -91),
             torch.full((32,), 2.0 ** -90), -torch.full((32,), 2.0 ** -90), torch.full((32,), 1e-40),
             torch.cat([torch.tensor([float("inf")]), torch.ones(31)]),
             torch.cat([torch.ones(31), torch.tensor([float("-inf")])]),
             torch.cat([torch.ones(17), torch.tensor([float("nan")]), torch.ones(14)]),
             torch.cat([torch.tensor([float("nan"), float("inf")]), torch.zeros(30)])]
    for i, k in enumerate(kinds):
        flat[i * 5 % flat.shape[0]] = k.to(BF)
    return x


def slots(kind, T, n, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "rows":
        return None
    if kind == "random":
        return torch.randperm(n, generator=g)[:T].to(torch.int32)
    if kind == "run":                          # a prompt's chunk that begins inside a unit
        return torch.arange(5, 5 + T, dtype=torch.int32)
    s = torch.randperm(n, generator=g)[:T].to(torch.int32)
    s[::3] = -1
    if T > 4:
        s[4] = -2 ** 31
    return s


def check(dims, k, v, slot, page, pages, seed=0, views=None):
    T, h, d = (k if k is not None else v).shape
    U = page // 16
    start = torch.randint(0, 256, (pages, h, U, 18 * d), generator=torch.Generator().manual_seed(seed), dtype=torch.uint8)
    want = start.numpy().copy()
    at = slot.tolist() if slot is not None else list(range(T))
    kv4.store(want, k, v, at)
    cache = start.to(DEV)
    dk, dv = views if views else (x.to(DEV) if x is not None else None for x in (k, v))
    ds = slot.to(DEV) if slot is not None else None
    gdn.gdn_kv4_store(dims, dk, dv, cache, slot=ds)
    assert np.array_equal(cache.cpu().numpy(), want)
    for dt in (torch.float32, BF):
        ko, vo = (torch.full((T, h, d), 7.0, dtype=dt, device=DEV) for _ in range(2))
        gdn.gdn_kv4_load(dims, cache, ko if k is not None else None, vo if v is not None else None, slot=ds)
        for x, got in ((k, ko), (v, vo)):
            if x is None:
                assert (got == 7.0).all()
                continue
            val = kv4.quantise(x)[2]
            for i, r in enumerate(at):
                if r < 0:
                    val[i] = 0
            torch.testing.assert_close(got.cpu(), val.to(torch.float32).to(dt), rtol=0, atol=0, equal_nan=True)
    return cache


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("h,page,T", [(1, 16, 1), (2, 64, 15), (3, 16, 16), (2, 32, 17), (1, 256, 70), (8, 128, 33)])
@pytest.mark.parametrize("kind", ["rows", "random", "run", "some"])
def test_rows_go_in_and_come_out(d, h, page, T, kind):
    dims = gdn.make_attn_dims(h_q=h, h_kv=h, d=d, rot=0)
    pages = (T + 5) // page + 2
    check(dims, special(T, h, d, 1), special(T, h, d, 2), slots(kind, T, pages * page, 3), page, pages, seed=d + T)


def test_every_ratio_to_the_extreme():
    # all significands of the extreme by all of a smaller number, 0 to 8 exponents below it, of
    # both signs: ties and what lies next to them, at exponents all over the range
    m = torch.arange(128, 256, dtype=torch.float64)
    x = (m[:, None] * 2.0 ** -torch.arange(9.0)).flatten()
    x = torch.cat([x, -x])                                              # [2304], 31 to a group
    x = torch.cat([x, torch.zeros(-len(x) % 31)]).view(1, -1, 31)
    big = m[:, None, None].expand(-1, x.shape[1], 1)
    x = x.expand(128, -1, -1).clamp(-big, big)                          # no larger than the extreme
    g = torch.Generator().manual_seed(7)
    by = 2.0 ** torch.randint(-80, 120, (*x.shape[:2], 1), generator=g)
    for sign in (1, -1):
        groups = (torch.cat([sign * big, x], -1) * by).view(-1, 32)
        groups = torch.cat([groups, torch.zeros(-len(groups) % 2, 32)])
        k = groups.view(-1, 1, 64).to(BF)
        assert torch.equal(k.double().view(-1, 32), groups)
        dims = gdn.make_attn_dims(h_q=1, h_kv=1, d=64, rot=0)
        T = len(k)
        cache = torch.zeros(-(-T // 256), 1, 16, 18 * 64, dtype=torch.uint8, device=DEV)
        gdn.gdn_kv4_store(dims, k.to(DEV), k.to(DEV), cache)
        ko, vo = (torch.empty(T, 1, 64, dtype=torch.float32, device=DEV) for _ in range(2))
        gdn.gdn_kv4_load(dims, cache, ko, vo)
        want = kv4.quantise(k)[2]
        assert torch.equal(ko.cpu().double(), want) and torch.equal(vo.cpu().double(), want)


def test_runs_broken_in_the_middle_and_pages_out_of_order():
    dims = gdn.make_attn_dims(h_q=2, h_kv=2, d=128, rot=0)
    T, page = 100, 16
    order = torch.tensor([5, 2, 9, 0, 7, 3, 8, 1])
    t = torch.arange(T) + 3
    s = (order[t // page] * page + t % page).to(torch.int32)
    check(dims, rows(T, 2, 128, 1), rows(T, 2, 128, 2), s, page, 10)
    s[[40, 41]] = s[[41, 40]]
    s[60] = -1
    check(dims, rows(T, 2, 128, 3), rows(T, 2, 128, 4), s, page, 10)


def test_one_of_k_and_v_and_strided_views():
    dims = gdn.make_attn_dims(h_q=2, h_kv=2, d=64, rot=0)
    k, v = rows(20, 2, 64, 1), rows(20, 2, 64, 2)
    check(dims, k, None, None, 32, 1)
    check(dims, None, v, slots("run", 20, 64, 0), 32, 2)
    # halves of a projection's output, heads apart
    big = torch.full((20, 5, 2, 72), float("nan"), dtype=BF, device=DEV)
    big[:, 1, :, :64], big[:, 3, :, :64] = k.to(DEV), v.to(DEV)
    check(dims, k, v, slots("random", 20, 64, 5), 32, 2, views=(big[:, 1, :, :64], big[:, 3, :, :64]))


def test_rows_out_of_range_are_named_and_left():
    dims = gdn.make_attn_dims(h_q=1, h_kv=1, d=64, rot=0)
    k = rows(3, 1, 64, 0).to(DEV)
    cache = torch.zeros(2, 1, 1, 18 * 64, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    s = torch.tensor([32, 2 ** 31 - 1, 31], dtype=torch.int32, device=DEV)
    gdn.gdn_kv4_store(dims, k, k, cache, slot=s, device_status=status)
    assert gdn.gdn_read_device_status(status) == gdn.GDN_ERR_DEVICE_BOUNDS
    want = np.zeros((2, 1, 1, 18 * 64), np.uint8)
    kv4.store(want, k.cpu(), k.cpu(), [-1, -1, 31])
    assert np.array_equal(cache.cpu().numpy(), want)
    status.zero_()
    out = torch.full((3, 1, 64), 5.0, device=DEV)
    gdn.gdn_kv4_load(dims, cache, out, None, slot=s, device_status=status)
    assert gdn.gdn_read_device_status(status) == gdn.GDN_ERR_DEVICE_BOUNDS
    assert (out[:2] == 0).all() and torch.equal(out[2].cpu().double(), kv4.quantise(k[2].cpu())[2])


def test_rows_far_into_a_large_cache():
    # byte offsets past 32 bits: 2^22 rows of 2 heads of 256 are 4.8 GB
    dims = gdn.make_attn_dims(h_q=2, h_kv=2, d=256, rot=0)
    pages = 1 << 14
    cache = torch.zeros(pages, 2, 16, 18 * 256, dtype=torch.uint8, device=DEV)
    s = torch.tensor([pages * 256 - 1, 5, pages * 256 - 200], dtype=torch.int32, device=DEV)
    k, v = rows(3, 2, 256, 1), rows(3, 2, 256, 2)
    gdn.gdn_kv4_store(dims, k.to(DEV), v.to(DEV), cache, slot=s)
    ko, vo = (torch.empty(3, 2, 256, device=DEV) for _ in range(2))
    gdn.gdn_kv4_load(dims, cache, ko, vo, slot=s)
    assert torch.equal(ko.cpu().double(), kv4.quantise(k)[2]) and torch.equal(vo.cpu().double(), kv4.quantise(v)[2])
    want = np.zeros((1, 2, 16, 18 * 256), np.uint8)
    kv4.store(want, k[[0, 2]], v[[0, 2]], [255, 56])
    assert np.array_equal(cache[-1:].cpu().numpy(), want)
