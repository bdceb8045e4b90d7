"""Strided inputs of the attention calls' binding: a dimension of size one has
no stride that matters, whatever number stands there (a slice of a fused
projection, viewed as [B, 1, heads, d], has one that is not the tokens')."""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

BF = torch.bfloat16


class OnDevice:
    """A CPU tensor that says it is on a device: only shapes and strides are looked at."""
    is_cuda = True

    def __init__(self, t):
        self.t, self.dtype, self.shape = t, t.dtype, t.shape

    def stride(self):
        return self.t.stride()

    def numel(self):
        return self.t.numel()

    def data_ptr(self):
        return self.t.data_ptr()


def view(t, tokens, heads, d):
    at, st, sh = gdn._view(OnDevice(t), "x", tokens, heads, d)
    assert at == t.data_ptr()
    return st, sh


def test_one_step_of_a_fused_projection():
    fused = torch.zeros(5, 3 * 256 + 64, dtype=BF)
    x = fused[:, 256:512].view(5, 1, 4, 64)
    assert x.stride() == (832, 256, 64, 1)          # the middle one is not a token's distance
    assert view(x, 5, 4, 64) == (832, 64)
    assert view(fused[:, 256:512].view(5, 4, 64), 5, 4, 64) == (832, 64)
    kv = torch.zeros(6, 2, 4, 64, dtype=BF)
    assert view(kv[:, 0][:, None], 6, 4, 64) == (512, 64)
    assert view(kv[:, 1][None], 6, 4, 64) == (512, 64)
    assert view(torch.zeros(3, 2, 4, 64, dtype=BF), 6, 4, 64) == (256, 64)


def test_one_token_or_one_head_has_no_stride():
    odd = torch.zeros(2, 4 * 64 + 4, dtype=BF)[:, :256].view(2, 4, 64)[:1]
    assert odd.stride()[0] == 260
    assert view(odd, 1, 4, 64) == (0, 64)
    assert view(odd[None], 1, 4, 64) == (0, 64)
    head = torch.zeros(7, 3, 64 + 8, dtype=BF).as_strided((7, 1, 64), (72, 9, 1))
    assert view(head, 7, 1, 64) == (72, 0)
    assert view(head[:, None], 7, 1, 64) == (72, 0)


def test_uneven_tokens_are_refused():
    x = torch.zeros(4, 3, 2, 64, dtype=BF)[:, :2]    # two of three: 2 apart, then 4
    with pytest.raises(ValueError):
        view(x, 8, 2, 64)
    with pytest.raises(ValueError):
        view(torch.zeros(4, 2, 64, dtype=BF).transpose(1, 2), 4, 2, 64)
    assert view(torch.zeros(2, 1, 3, 2, 64, dtype=BF), 6, 2, 64) == (128, 64)


@pytest.mark.gpu
def test_a_gate_inside_a_fused_projection():
    B, h, d = 3, 4, 64
    dims = gdn.make_attn_dims(h_q=h, h_kv=2, d=d, rot=0)
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    fused, kc, vc = r(B, 2 * h * d + 64), r(4, 16, 2, d), r(4, 16, 2, d)
    q, pages = r(B, 1, h, d), torch.arange(4, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.gdn_attn_decode_shared_workspace_bytes(dims, B), dtype=torch.uint8, device="cuda")
    out = []
    for gate in (fused[:, h * d:2 * h * d].contiguous().view(B, 1, h, d), fused[:, h * d:2 * h * d].view(B, 1, h, d)):
        o = torch.zeros_like(q)
        gdn.gdn_attn_decode_shared(dims, q, kc, vc, pages, 50, None, None, o, ws, gate=gate)
        out.append(o)
    assert torch.equal(*out) and out[0].abs().sum() > 0
