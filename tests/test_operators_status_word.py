"""The status word that calls without one share: threads whose first calls meet get
the same one.  torch's device calls are stood in for: no GPU is needed."""
import threading
import time

import torch

from block_scaled_grouped_gb300 import operators as ops


class OnGpu:
    device = torch.device("cpu")

    def get_device(self):
        return 0


def test_first_calls_of_many_threads_share_one_word(monkeypatch):
    monkeypatch.setattr(ops, "_status_words", {})
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: time.sleep(0.05))     # others run meanwhile
    got, together = [], threading.Barrier(8)

    def call():
        together.wait()
        got.append(ops._status_of(OnGpu(), None))

    threads = [threading.Thread(target=call) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    word, address = ops._status_words[0]
    assert len(got) == 8 and set(got) == {address} and word.data_ptr() == address
