"""gdn_attn_decode_kv4 through tables that are wider than the sequences: the entries behind a
sequence's end do not matter, and only the order of a row's sums may follow the width.

Two orders of a row's sums differ by at most their own fp32 roundings, far below a bf16 step, and
the result is rounded to bf16 in both: by one step of it at most, 2^-7 of the result, or of what
cancels, 2^-16 of the largest value."""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn
from test_attn_kv4_gpu import DEV, build, call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hk,S", [(64, 8, 1, 1), (128, 8, 2, 2), (256, 16, 2, 1)])
@pytest.mark.parametrize("lens", [[833], [3000, 40], [700, 1, 0, 90]])
def test_a_wider_table_gives_the_same(d, hq, hk, S, lens):
    x = build(len(lens), S, hq, hk, d, 16, lens, seed=d, gate=False)
    got = check(x)
    for width, entry in ((400, 0), (4096, -9), (60000, 2 ** 31 - 1)):
        table = torch.full((len(lens), width), entry, dtype=torch.int32, device=DEV)
        table[:, :x["table"].shape[1]] = x["table"]
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        y = dict(x, table=table)
        wide = call(y, status=status)
        assert gdn.gdn_read_device_status(status) == 0
        assert torch.equal(wide, call(y))      # equal calls, equal bits
        tol = 2 ** -7 * got.float().abs() + 2 ** -16 * 8
        assert ((wide.float() - got.float()).abs() <= tol).all()
