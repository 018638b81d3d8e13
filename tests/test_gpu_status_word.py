"""The operators' status word with several streams."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu


def crowded():
    """Slots that do not fit 256 rows."""
    return (torch.arange(600, dtype=torch.int32) % 8).view(300, 2).cuda()


def test_shared_word_is_read_after_every_stream():
    ids, side = crowded(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            bsgg.sort_tokens(ids, 8)                     # the stream's memory is there: no allocation waits
    torch.cuda.synchronize()
    assert bsgg.operators_status() == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                   # a tenth of a second
        bsgg.sort_tokens(ids, 8, m_pad=256)
    assert bsgg.operators_status() == 5
    assert bsgg.operators_status() == 0


def test_reports_are_seen_once_each():
    """Reading goes on while another stream's kernel reports: each report is seen
    by one of the reads."""
    ids, status, side = crowded(), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    lost = 0
    for i in range(2000):
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000 + 997 * (i % 50))  # reads are under way when the report comes
            bsgg.sort_tokens(ids, 8, m_pad=256, status=status)
            done = side.record_event()
        while True:
            finished = done.query()
            if bsgg.operators_status(status=status) == 5:
                break
            if finished:
                lost += 1
                break
        done.synchronize()
        bsgg.operators_status(status=status)
    assert lost == 0
