"""The weights' gradient of combine without the rows', where the rows themselves
take no gradient: against 64 bits, and the bits of the joint call."""
import math

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
import operator_refs as R
from test_gpu_tokens import DT, gen, ids_of, pitched

pytestmark = pytest.mark.gpu

CASES = [(1, 8, 1, 2, "bf16", "bf16"), (1, 7168, 8, 64, "bf16", "bf16"), (37, 264, 3, 5, "f16", "f32"), (100, 1032, 4, 8, "f32", "bf16"),
         (513, 4096, 2, 8, "bf16", "f16"), (60, 24, 8, 16, "f32", "f32"), (9, 2056, 32, 40, "bf16", "f32")]


@pytest.mark.parametrize("T,H,k,L,dk,yk", CASES)
def test_dweights_alone(T, H, k, L, dk, yk):
    ids = ids_of(T, L, k, H, T > 8)
    m_pad = bsgg.sort_rows(T * k, L)
    _, row_of_slot, slot_of_row, _ = R.sort_tokens(ids, L, m_pad)
    g = gen(T + H)
    d = torch.randn(m_pad, H, generator=g).to(DT[dk])
    d[torch.tensor(slot_of_row) < 0] = math.nan               # padding rows are not read
    dy = torch.randn(T, H, generator=g).to(DT[yk])
    rs = torch.tensor(row_of_slot, dtype=torch.int32).view(T, k)
    sr = torch.tensor(slot_of_row, dtype=torch.int32).cuda()
    args = (pitched(dy, 8), d.cuda(), rs.cuda(), sr)
    dd, sfd, dw = bsgg.combine_backward(*args, want_dd=False)
    assert dd is None and sfd is None and dw.shape == (T, k)
    r = rs.long()
    terms = torch.where((r >= 0)[..., None], d.double()[r.clamp(min=0)], torch.zeros((), dtype=torch.float64)) * dy.double()[:, None, :]
    # a thread's products one after the other, then the lanes' and the warps' sums
    assert ((dw.cpu().double() - terms.sum(-1)).abs() <= terms.abs().sum(-1) * (H / 32 + 8) * 2.0 ** -24).all()
    assert (dw.cpu()[rs < 0] == 0).all()
    assert torch.equal(bsgg.combine_backward(*args)[2], dw)


def test_a_gradient_has_to_be_wanted():
    z = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(bsgg.BsggError):
        bsgg.combine_backward(x, None, z, torch.zeros(128, dtype=torch.int32, device="cuda"), want_dweights=False, want_dd=False)
