"""A wait of the orthogonalisation that runs out is reported in the status word, whichever kernel gave up.
A debug setting makes the first CTA of the next such kernel wait for an arrival that never comes."""
import pytest
import torch

from _layers import randn

pytestmark = pytest.mark.gpu


# one kernel with one and with several CTAs a matrix; the first product on single CTAs (all of A, its blocks of
# 128, of 256) and on pairs, with one tile each and with several
@pytest.mark.parametrize("shape", [(1, 100, 100), (3, 120, 1024), (3, 1024, 120), (170, 60, 250), (1, 100, 1100), (1, 900, 700), (1, 950, 1300), (1, 900, 5000),
                                   (6, 1024, 1024), (40, 600, 700), (1, 2600, 2200)])
@pytest.mark.parametrize("stage", [0, 1])
def test_the_status_word(cuda_lib, shape, stage):
    rlk = cuda_lib
    g = randn(shape, 1)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = rlk.orthogonalise(g, status_word=word)
    torch.cuda.synchronize()
    assert word.item() == 0
    rlk.set_wait_limit(2_000_000)   # about a millisecond
    try:
        rlk.withhold_copy(stage)
        got = rlk.orthogonalise(g, status_word=word)
        torch.cuda.synchronize()
    finally:
        rlk.withhold_copy(-1)
        rlk.set_wait_limit(0)
    assert torch.isnan(got).any() and word.item() == rlk.STATUS_TIMEOUT | rlk.STATUS_NONFINITE
    word.zero_()
    assert torch.equal(rlk.orthogonalise(g, status_word=word), want) and word.item() == 0
