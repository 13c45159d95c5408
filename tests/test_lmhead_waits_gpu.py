"""The LM-head kernel's waits running out after its last copy was asked for (a few
tiles in all): the call reports it, its rows are NaN, the next call is clean."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


# a vocabulary of 19 tiles or more: the first CTA has one, and its K fits the ring
@pytest.mark.parametrize("T,H,V", [(64, 128, 5000), (100, 64, 4900), (128, 192, 5000)])
def test_few_tiles(cuda_lib, T, H, V):
    hidden, w, ids = workloads.lmhead_inputs(T, H, V, seed=3, device="cuda")
    want = cuda_lib.lmhead_logprob(hidden, w, ids, 0.7)
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    cuda_lib.set_wait_limit(2_000_000)   # about a millisecond
    try:
        cuda_lib.withhold_copy(0)
        lp, ent = cuda_lib.lmhead_logprob(hidden, w, ids, 0.7, status_word=st[:1])
        torch.cuda.synchronize()
    finally:
        cuda_lib.withhold_copy(-1)
        cuda_lib.set_wait_limit(0)
    assert int(st[0]) & cuda_lib.STATUS_TIMEOUT and torch.isnan(lp).all() and torch.isnan(ent).all()
    for _ in range(3):
        got = cuda_lib.lmhead_logprob(hidden, w, ids, 0.7, status_word=st[1:])
        assert int(st[1]) == 0 and all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(got, want))
