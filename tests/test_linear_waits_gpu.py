"""The linear layer's waits running out after the last copy was asked for: K is short
enough for the ring, so the producer has nothing left to do when the products give up.
The call returns once its copies are there, what depended on them is NaN, and the
next call is clean."""
import pytest
import torch

from _layers import randn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


# one tile a CTA, its K whole and split; pairs with one and with several tiles
@pytest.mark.parametrize("M,N,K", [(40, 64, 130), (100, 300, 512), (3000, 2816, 250), (6000, 5600, 128)])
@pytest.mark.parametrize("stage", [0, 1])
def test_short_k(cuda_lib, M, N, K, stage):
    x, w = randn((M, K), 1, BF), randn((N, K), 2, BF, 0.05)
    want = cuda_lib.linear(x, w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    cuda_lib.set_wait_limit(2_000_000)   # about a millisecond
    try:
        cuda_lib.withhold_copy(stage)
        got = cuda_lib.linear(x, w, out_dtype=torch.float32)
        torch.cuda.synchronize()
    finally:
        cuda_lib.withhold_copy(-1)
        cuda_lib.set_wait_limit(0)
    nan = torch.isnan(got)
    assert bool(nan[0, 0]) and torch.equal(got[~nan], want[~nan])
    for _ in range(3):
        assert torch.equal(cuda_lib.linear(x, w, out_dtype=torch.float32), want)
