"""gdn_moe_step where an activation between the two products is near the end of
fp32's range or beyond it.  Beyond it the token's results are infinite with
their sign; within it, but past the largest bf16, they are what the formula
gives.  The other tokens keep their bits.

Tolerance of the second: the activation is the one term that counts (the next is
2^-70 of it).  Its parts hold 16 bits (bf16 result) or 24 (fp32), the products
and sums are fp32 with an error below 2^-18, and a bf16 result is rounded:
2^-15 + 2^-18 (+ 2^-8).
"""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
from test_moe_gpu import BF, F32, call, inputs

pytestmark = pytest.mark.gpu
T, H, I = 3, 64, 16


def layer(shared, gate, up):
    """Weights whose gate and up rows 3 read element 0 of x, by these factors."""
    w = inputs(T, H, I, 2, I if shared else 0, seed=5, gate=False)
    w["x"][:, 0] = 0
    w["wr"][:, 0] = 0
    gu, dn = (w["sgu"], w["sdn"]) if shared else (w["gu"][1], w["dn"][1])
    gu[3, 0], gu[I + 3, 0] = gate, up
    dn[dn == 0] = 0.5
    return w, dn[:, 3].double(), gdn.make_moe_dims(hidden=H, inter=I, experts=2, top_k=2, shared_inter=I if shared else 0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shared", [False, True])
def test_an_activation_beyond_the_range_is_infinite(dtype, shared):
    w, dn, dims = layer(shared, 2.0 ** 45, 2.0 ** 45)
    want, _, _ = call(dims, w, dtype)
    assert want.isfinite().all()
    w["x"][1, 0] = 2.0 ** 24                             # gate and up 2^69 each
    y, _, _ = call(dims, w, dtype)
    assert torch.equal(y[1].double().cpu(), torch.sign(dn) * float("inf"))
    assert torch.equal(y[[0, 2]], want[[0, 2]])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_an_activation_that_bf16_would_round_to_infinity(dtype):
    gate, up = 2.0 ** 40 * (1 + 2 / 128), 2.0 ** 40 * (1 - 4 / 256)
    w, dn, dims = layer(True, gate, up)
    w["x"][1, 0] = 2.0 ** 24
    act = gate * up * 2.0 ** 48                          # in fp32's range, nearer to 2^128 than to the largest bf16
    assert torch.tensor(act, dtype=F32).isfinite() and torch.tensor(act, dtype=F32).to(BF).isinf()
    y, _, _ = call(dims, w, dtype)
    ref = act * dn
    tol = (2.0 ** -15 + 2.0 ** -18 + (2.0 ** -8 if dtype == BF else 0.0)) * ref.abs()
    assert ((y[1].double().cpu() - ref).abs() <= tol).all()
