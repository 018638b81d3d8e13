"""sort_tokens from two host threads at once, over numbers of experts whose counts need
different amounts of shared memory beyond the default limit."""
import threading

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots,times", [(64, 60000), (9000, 20000)])
def test_numbers_of_experts_in_two_threads(slots, times):
    lib, codes, maps = bsgg.lib(), {}, {}
    torch.cuda.synchronize()

    def calls(L):
        s = torch.cuda.Stream()
        ids = (torch.arange(slots, dtype=torch.int32) * 7 % L).view(-1, 1).cuda()
        t = bsgg.sort_tokens(ids, L)
        for v in t:
            v.fill_(-7)
        ws = torch.empty(max(1, lib.bsgg_sort_workspace_bytes(slots, L) // 4), dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        args = (slots, L, t.slot_of_row.numel(), ids.data_ptr(), None, t.padded_offsets.data_ptr(), t.row_of_slot.data_ptr(),
                t.slot_of_row.data_ptr(), t.prob.data_ptr(), t.rows_used.data_ptr(), ws.data_ptr(), status.data_ptr(), s.cuda_stream)
        codes[L] = [lib.bsgg_sort_tokens(*args) for _ in range(times)]
        s.synchronize()
        maps[L] = (ids, t)

    threads = [threading.Thread(target=calls, args=(L,)) for L in (640, 1024)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted((L, len(c), sum(c)) for L, c in codes.items()) == [(640, times, 0), (1024, times, 0)] and len(maps) == 2
    for L, (ids, t) in maps.items():
        assert all(torch.equal(a, b) for a, b in zip(t, bsgg.sort_tokens(ids, L)))
