"""The binding's calls refuse tensors of another device than the first one's, each of
their tensors in turn.  Stand-ins for CUDA tensors: no GPU is needed."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
from block_scaled_grouped_gb300 import operators as ops

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class OnGpu:
    """What the binding asks of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), 0

    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


T, H, L, K, M, N = 4, 64, 8, 2, 128, 16
CALLS = {
    "route": (lambda t: bsgg.route(t["logits"], K, ids=t["ids"], weights=t["weights"]),
              dict(logits=(F32, T, L), ids=(I32, T, K), weights=(F32, T, K))),
    "route_backward": (lambda t: bsgg.route_backward(t["logits"], t["ids"], t["weights"], t["dweights"],
                                                     row_of_slot=t["row_of_slot"], dlogits=t["dlogits"]),
                       dict(logits=(F32, T, L), ids=(I32, T, K), weights=(F32, T, K), dweights=(F32, M),
                            row_of_slot=(I32, T, K), dlogits=(F32, T, L))),
    "sort_tokens": (lambda t: bsgg.sort_tokens(t["ids"], L, weights=t["weights"], status=t["status"]),
                    dict(ids=(I32, T, K), weights=(F32, T, K), status=(I32, 1))),
    "dispatch": (lambda t: bsgg.dispatch(t["x"], t["row_of_slot"], t["slot_of_row"]),
                 dict(x=(BF, T, H), row_of_slot=(I32, T, K), slot_of_row=(I32, M))),
    "combine": (lambda t: bsgg.combine(t["d"], t["row_of_slot"], weights=t["weights"], residual=t["residual"], out=t["out"]),
                dict(d=(BF, M, H), row_of_slot=(I32, T, K), weights=(F32, T, K), residual=(BF, T, H), out=(BF, T, H))),
    "combine_backward": (lambda t: bsgg.combine_backward(t["dy"], t["d"], t["row_of_slot"], t["slot_of_row"],
                                                         weights=t["weights"]),
                         dict(dy=(BF, T, H), d=(BF, M, H), row_of_slot=(I32, T, K), slot_of_row=(I32, M),
                              weights=(F32, T, K))),
    "linear": (lambda t: bsgg.linear(t["x"], t["w"], bias=t["bias"], residual=t["residual"], out=t["out"], status=t["status"]),
               dict(x=(BF, T, H), w=(BF, N, H), bias=(F32, N), residual=(BF, T, N), out=(BF, T, N), status=(I32, 1))),
    "linear_backward": (lambda t: bsgg.linear_backward(t["dy"], t["x"], t["w"], z=t["z"], activation="silu", dw=t["dw"],
                                                       status=t["status"]),
                        dict(dy=(BF, T, N), x=(BF, T, H), w=(BF, N, H), z=(BF, T, N), dw=(F32, N, H), status=(I32, 1))),
}
EACH = [(call, name) for call, (_, tensors) in CALLS.items() for name in tensors]


@pytest.fixture(autouse=True)
def a_gpu(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)


@pytest.mark.parametrize("call,name", EACH)
def test_another_device_is_refused(call, name):
    run, tensors = CALLS[call]
    t = {n: OnGpu(*spec) for n, spec in tensors.items()}
    t[name].index = 1
    with pytest.raises(ValueError, match="cuda:1"):
        run(t)


def test_absent_tensors_pass():
    assert ops._handle(None, OnGpu(BF, 1), None, OnGpu(BF, 1)) == 0
