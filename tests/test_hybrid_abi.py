"""Host-side checks of the attention-layer and expert-layer calls: refusals
before anything touches a device, empty calls, workspace sizes.  No call here
reaches the GPU."""
import ctypes

import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
from gated_deltanet_linear_06_gb300 import build as gbuild

FAKE = 0x10000          # aligned, never dereferenced on these paths
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdn.lib()


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _prep(L, dims, **kw):
    a = dict(tokens=4, q=FAKE, q_st=4096, q_sh=256, k=FAKE, k_st=512, k_sh=256, v=FAKE, v_st=512, v_sh=256,
             q_w=FAKE, k_w=FAKE, inv_freq=FAKE, axis=None, pos=FAKE, slot=FAKE, rows=64, q_out=FAKE,
             k_cache=FAKE, v_cache=FAKE, status=None, stream=None)
    a.update(kw)
    return L.gdn_attn_prep(_ref(dims), *a.values())


def _shared(L, dims, **kw):
    a = dict(page=64, n_pages=100, batch=2, steps=1, q=FAKE, k_cache=FAKE, v_cache=FAKE, prefix_pages=FAKE,
             prefix_len=100, tail_pages=FAKE, tail_width=2, tail_len=FAKE, gate=None, g_st=0, g_sh=0, out=FAKE,
             ws=0x100000, ws_bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    return L.gdn_attn_decode_shared(_ref(dims), *a.values())


def _moe(L, dims, **kw):
    a = dict(tokens=2, x=FAKE, w_router=FAKE, w_gate_up=FAKE, w_down=FAKE, s_gu=None, s_d=None, s_g=None,
             y=FAKE, dtype=0, ids=None, wts=None, ws=0x100000, ws_bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    return L.gdn_moe_step(_ref(dims), *a.values())


@pytest.mark.parametrize("bad,want", [
    (dict(h_q=0), INVALID), (dict(h_kv=3), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=0), INVALID),
    (dict(rot=8), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(rot=512), INVALID), (dict(n_axes=0), INVALID),
    (dict(n_axes=5), UNSUPPORTED), (dict(rope_pairs=2), INVALID), (dict(norm_eps=float("nan")), INVALID),
    (dict(norm_eps=-1.0), INVALID), (dict(scale=float("inf")), INVALID), (dict(h_q=2048, h_kv=2048), UNSUPPORTED)])
def test_attention_dims_are_checked(L, bad, want):
    d = gdn.make_attn_dims(**bad)
    assert _prep(L, d) == want
    assert _shared(L, d) == want
    assert gdn.gdn_attn_decode_shared_workspace_bytes(d, 2) == 0
    assert _prep(L, None) == INVALID and _shared(L, None) == INVALID


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), INVALID), (dict(q=FAKE + 2), INVALID),
    (dict(q_out=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=FAKE + 8), INVALID),
    (dict(q_st=4097), INVALID), (dict(k_sh=-8), INVALID), (dict(inv_freq=None), INVALID),
    (dict(pos=None), INVALID), (dict(slot=None, rows=3), INVALID), (dict(rows=-1), INVALID),
    (dict(status=FAKE + 2), INVALID), (dict(q_w=FAKE + 4), INVALID), (dict(slot=FAKE + 4), INVALID)])
def test_prep_refusals(L, bad, want):
    assert _prep(L, gdn.make_attn_dims(), **bad) == want


def test_prep_needs_axes_and_empty_calls_do_nothing(L):
    assert _prep(L, gdn.make_attn_dims(n_axes=3), axis=None) == INVALID
    assert _prep(L, gdn.make_attn_dims(), tokens=0, q=None) == OK
    assert _prep(L, gdn.make_attn_dims(), q=None, k=None, v=None) == OK


@pytest.mark.parametrize("bad,want", [
    (dict(page=0), INVALID), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(batch=-1), INVALID),
    (dict(batch=1025), UNSUPPORTED), (dict(steps=0), INVALID), (dict(steps=9), UNSUPPORTED),
    (dict(prefix_len=-1), INVALID), (dict(prefix_len=1 << 31), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(n_pages=1 << 31), UNSUPPORTED), (dict(tail_width=-1), INVALID), (dict(tail_width=1 << 30), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=None), INVALID), (dict(k_cache=None), INVALID),
    (dict(prefix_pages=None), INVALID), (dict(tail_pages=None), INVALID), (dict(tail_len=None), INVALID),
    (dict(gate=FAKE, g_st=4, g_sh=256), INVALID), (dict(gate=FAKE + 2), INVALID),
    (dict(status=FAKE + 1), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=0x100010), WORKSPACE),
    (dict(ws_bytes=100), WORKSPACE)])
def test_shared_refusals(L, bad, want):
    assert _shared(L, gdn.make_attn_dims(), **bad) == want


def test_shared_limits_and_empty_batch(L):
    assert _shared(L, gdn.make_attn_dims(), batch=0, q=None, ws=None) == OK
    # steps * group rows share one tile of 128
    d = gdn.make_attn_dims(h_q=34, h_kv=2)
    assert gdn.gdn_attn_decode_shared_workspace_bytes(d, 1, 7) > 0
    assert gdn.gdn_attn_decode_shared_workspace_bytes(d, 1, 8) == 0
    assert _shared(L, d, steps=8) == UNSUPPORTED


@pytest.mark.parametrize("bad,want", [
    (dict(hidden=0), INVALID), (dict(inter=-8), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=300), INVALID), (dict(shared_inter=-8), INVALID), (dict(hidden=2052), UNSUPPORTED),
    (dict(inter=500), UNSUPPORTED), (dict(shared_inter=4), UNSUPPORTED), (dict(hidden=16392), UNSUPPORTED),
    (dict(experts=1025), UNSUPPORTED), (dict(top_k=33), UNSUPPORTED)])
def test_moe_dims_are_checked(L, bad, want):
    d = gdn.make_moe_dims(**bad)
    assert _moe(L, d) == want
    assert gdn.gdn_moe_step_workspace_bytes(d, 2) == 0
    assert _moe(L, None) == INVALID


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=-1), INVALID), (dict(tokens=65), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(x=None), INVALID),
    (dict(w_router=FAKE + 8), INVALID), (dict(w_gate_up=None), INVALID), (dict(w_down=None), INVALID),
    (dict(y=None), INVALID), (dict(ids=FAKE + 4), INVALID), (dict(wts=FAKE + 4), INVALID),
    (dict(status=FAKE + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=0x100080), WORKSPACE),
    (dict(ws_bytes=16), WORKSPACE)])
def test_moe_refusals(L, bad, want):
    assert _moe(L, gdn.make_moe_dims(), **bad) == want


def test_moe_shared_expert_needs_its_weights_and_empty_calls_do_nothing(L):
    d = gdn.make_moe_dims(shared_inter=256)
    assert _moe(L, d) == INVALID
    assert _moe(L, d, s_gu=FAKE, s_d=FAKE, s_g=FAKE + 2) == INVALID
    assert _moe(L, d, tokens=0, x=None, ws=None) == OK


def test_workspaces_grow_with_their_problem(L):
    a = gdn.make_attn_dims()
    w = [gdn.gdn_attn_decode_shared_workspace_bytes(a, b, s) for b, s in ((1, 1), (64, 1), (64, 4), (1024, 8))]
    assert 0 < w[0] <= w[1] <= w[2] <= w[3]
    m = [gdn.gdn_moe_step_workspace_bytes(gdn.make_moe_dims(), t) for t in (1, 8, 64)]
    assert 0 < m[0] <= m[1] <= m[2]


def test_the_binding_refuses_what_the_call_would_misread():
    d = gdn.make_attn_dims(h_q=2, h_kv=1, d=64, rot=32)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):      # host tensors
        gdn.gdn_attn_prep(d, x, None, None, None, None, None, None, None, x, None, None)
    kv = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):      # caches that differ
        gdn.gdn_attn_decode_shared(d, x[None], kv, kv[:1], None, 0, None, None, x, x)
    with pytest.raises(ValueError):      # fewer pages than the prefix has
        gdn.gdn_attn_decode_shared(d, x[None], kv, kv, torch.zeros(1, dtype=torch.int32), 17, None, None, x, x)
    with pytest.raises(ValueError):      # an output type the call does not write
        gdn.gdn_moe_step(gdn.make_moe_dims(), x, x, x, x, x.half(), x)
