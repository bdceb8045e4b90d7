"""gdn_attn_decode_kv4 where V's magnitudes step up within a warp's share of the tokens.

As many jobs as several GPUs have warps: shares hold whole jobs, so that what a share has
summed meets values of another size.  All sequences read one sequence's pages.  The
tolerance is test_attn_kv4_gpu's."""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
from test_attn_kv4_gpu import BF, DEV, build, call, values

pytestmark = pytest.mark.gpu
JOBS = 4096


def many(S, G, d, n, k, v, seed, std=1.0):
    """JOBS jobs of S steps and G heads over the same n tokens of k and v ([n, 8, d])."""
    x = build(1, S, 8 * G, 8, d, 16, [n], seed=seed, gate=False)
    gdn.gdn_kv4_store(x["dims"], k.to(BF).to(DEV), v.to(BF).to(DEV), x["cache"], slot=x["slot"].to(DEV))
    B = JOBS // 8
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(B, S, 8 * G, d, generator=g) * std).to(BF).to(DEV)
    return dict(x, q=q, table=x["table"].expand(B, -1).contiguous(), lens=x["lens"].expand(B).contiguous())


def against_the_formula(x, S, n):
    """Largest error in units of the tolerance, over all jobs."""
    k, v = values(x)
    B, _, hq, d = x["q"].shape
    hk = x["dims"].h_kv
    q = x["q"].double().unflatten(2, (hk, hq // hk))
    got = call(x).double().unflatten(2, (hk, hq // hk))
    most = v.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
    worst = 0.0
    for i in range(S):
        m = n - S + 1 + i
        p = torch.softmax(torch.einsum("nhd,bhgd->bhgn", k[:m], q[:, i]) * d ** -0.5, -1)
        want = torch.einsum("bhgn,nhd->bhgd", p, v[:m])
        size = torch.einsum("bhgn,nhd->bhgd", p, v[:m].abs() + 2 ** -6 * most[:m])
        err = (got[:, i] - want).abs() / (2 ** -8 * want.abs() + 2 ** -10 * size + 1e-30)
        worst = max(worst, err.nan_to_num(nan=float("inf")).max().item())
    return worst


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("S,G", [(1, 4), (4, 4)])
@pytest.mark.parametrize("low,high", [(None, 40), (None, 100), (-60, 70), (-85, 120)])
def test_tokens_before_a_large_step_in_values_stay_in_the_sum(d, S, G, low, high):
    n = 200
    g = torch.Generator().manual_seed(d)
    k, v = torch.randn(n, 8, d, generator=g), torch.randn(n, 8, d, generator=g)
    v[:100] *= 0.0 if low is None else 2.0 ** low
    v[100:] *= 2.0 ** high
    assert against_the_formula(many(S, G, d, n, k, v, seed=d + S), S, n) <= 1
