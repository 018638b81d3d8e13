"""Sorts of so many slots that a block's ranks pass 16 bits: each against the
definition, expert by expert."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu


def check(ids, L):
    n = ids.numel()
    w = torch.rand(ids.shape, device="cuda")
    tm = bsgg.sort_tokens(ids, L, weights=w)
    assert bsgg.operators_status() == 0
    flat, row_of_slot, at = ids.reshape(-1), tm.row_of_slot.reshape(-1), 0
    for e in range(L):
        mine = torch.nonzero(flat == e)[:, 0].to(torch.int32)      # in order of slot
        c = mine.numel()
        end = at + -(-c // 128) * 128
        assert torch.equal(tm.slot_of_row[at:at + c], mine)
        assert torch.equal(row_of_slot[mine.long()], torch.arange(at, at + c, dtype=torch.int32, device="cuda"))
        assert torch.equal(tm.prob[at:at + c], w.reshape(-1)[mine.long()])
        assert (tm.slot_of_row[at + c:end] == -1).all() and (tm.prob[at + c:end] == 0).all()
        if e + 1 < L:
            assert tm.padded_offsets[e].item() == end
        at = end
        del mine
    m_pad = tm.slot_of_row.numel()
    assert tm.rows_used.item() == at and tm.padded_offsets[L - 1].item() == m_pad
    assert (tm.slot_of_row[at:] == -1).all()
    out = (flat < 0) | (flat >= L)
    assert (row_of_slot[out] == -1).all() and int((row_of_slot >= 0).sum()) == n - int(out.sum())


@pytest.mark.parametrize("n", [9699328, 9699329, 12000001])
def test_one_expert(n):
    """128 and 129 steps a warp, all slots of one expert."""
    check(torch.zeros(n, 1, dtype=torch.int32, device="cuda"), 1)


@pytest.mark.parametrize("L", [2, 1024])
def test_two_experts_of_many(L):
    """Two experts take every slot, eleven twelfths and one."""
    T = 6000000
    ids = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    ids[::6, 1] = L - 1
    check(ids, L)


def test_runs_of_one_expert_and_masked_slots():
    """Slots that come expert by expert, every fifth one masked."""
    T, L = 5000000, 3
    ids = (torch.arange(4 * T, device="cuda") * L // (4 * T)).to(torch.int32)
    ids[::5] = -1
    check(ids.view(T, 4), L)


def test_two_hundred_million_slots():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randint(-1, 4, (25000000, 8), generator=g, device="cuda", dtype=torch.int32)
    check(ids, 3)
