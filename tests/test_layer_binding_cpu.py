"""The layers' binding on the host: what it refuses before the library is called.
Tensors that say that they are on a CUDA device stand in for such ones; launches are
made to fail."""
import pytest
import torch

import entropy_logits_bf16_gb300 as rlk

BF, F32 = torch.bfloat16, torch.float32


class OnCuda(torch.Tensor):
    is_cuda = property(lambda self: True)


def cuda(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnCuda)


@pytest.fixture(autouse=True)
def lib(monkeypatch):
    rlk.build()
    lib = rlk.load()
    monkeypatch.setattr(rlk, "_stream", lambda device: 0)
    lib.rlk_debug_inject_launch_failures(1000)
    yield lib
    lib.rlk_debug_inject_launch_failures(0)


def test_workspaces_on_the_host_are_refused():
    dy, x, w, r = cuda(4, 64), cuda(4, 64), cuda(64), cuda(4)
    off, lp = cuda(5, dtype=torch.int32), cuda(50)
    for call in (lambda ws: rlk.norm_backward(dy, x, w, None, r, kind=rlk.NORM_RMS, workspace=ws),
                 lambda ws: rlk.preference_loss(lp, None, off, workspace=ws)):
        with pytest.raises(rlk.RlkError):      # on the device: on to the launch, which fails
            call(cuda(1 << 16, dtype=torch.uint8))
        with pytest.raises(ValueError):
            call(torch.zeros(1 << 16, dtype=torch.uint8))
