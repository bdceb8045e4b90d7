"""The attention and expert calls at the limits that include/gdn.h states:
batches whose tails' costs are summed in several passes, and rows of the
router and of the expert products that take many.  Tolerances as in the
operators' own tests, whose definitions these use."""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
import test_attn_shared_gpu as attn
import test_moe_gpu as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,S,hq,hk,prefix,hi", [
    (384, 1, 2, 1, 30, 40), (385, 1, 2, 2, 0, 30), (769, 2, 1, 1, 200, 20), (1024, 1, 2, 1, 100, 140),
    (1024, 8, 1, 1, 20, 12)])
def test_large_batches(B, S, hq, hk, prefix, hi):
    g = torch.Generator().manual_seed(B)
    tails = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    dims = gdn.make_attn_dims(h_q=hq, h_kv=hk, d=64, rot=0)
    attn.check(dims, attn.build(B, S, hq, hk, 64, 16, prefix, tails, seed=B + S))


def test_empty_tails_between_long_ones():
    tails = [0] * 1024
    tails[3], tails[500], tails[1023] = 700, 129, 1
    dims = gdn.make_attn_dims(h_q=2, h_kv=1, d=64, rot=0)
    attn.check(dims, attn.build(1024, 1, 2, 1, 64, 16, 0, tails, seed=4))


def test_most_rows_of_a_sequence():
    # steps * group = 128 rows of one job
    dims = gdn.make_attn_dims(h_q=16, h_kv=1, d=128, rot=0)
    attn.check(dims, attn.build(5, 8, 16, 1, 128, 32, 140, [8, 300, 0, 17, 128], seed=9))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,I,E,k,Is", [
    (1, 16384, 16, 5, 2, 8), (9, 8200, 24, 4, 2, 0), (3, 16, 16384, 3, 2, 16384), (64, 4096, 8, 20, 3, 8)])
def test_long_rows_of_an_expert(T, H, I, E, k, Is, dtype):
    moe.check(moe.inputs(T, H, I, E, Is, seed=H + I), I, k, True, dtype)


def test_most_experts_and_most_chosen():
    moe.check(moe.inputs(64, 64, 8, 1024, 0, seed=2), 8, 32, False, torch.float32)
