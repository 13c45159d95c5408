"""The expiry path of the layers' bounded device waits: a debug setting makes the
first CTA wait for an arrival that never comes (nothing is left in flight) and
shortens the limit.
The call returns, what depended on it is NaN and the rest keeps its bits;
the next call is clean."""
import pytest
import torch

from _layers import randn, rows

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def timed_out(rlk, stage, call):
    torch.cuda.synchronize()
    rlk.set_wait_limit(2_000_000)   # about a millisecond
    try:
        rlk.withhold_copy(stage)
        out = call()
        torch.cuda.synchronize()
    finally:
        rlk.withhold_copy(-1)
        rlk.set_wait_limit(0)
    return out


@pytest.mark.parametrize("H", [64, 4096, 5003, 9000])
def test_norm(cuda_lib, H):
    T = 2000
    x, dy, w = rows(T, H, BF, 1), randn((T, H), 2, BF), randn((H,), 3)
    y, mean, rstd = cuda_lib.norm(x, w)
    want = cuda_lib.norm_backward(dy, x, w, mean, rstd)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad, _, bad_r = timed_out(cuda_lib, 0, lambda: cuda_lib.norm(x, w, status_word=st))   # rows of 64: a group has one row only
    nan = torch.isnan(bad_r)
    assert int(st) & cuda_lib.STATUS_TIMEOUT and 0 < int(nan.sum()) < T
    assert torch.isnan(bad[nan]).all() and torch.equal(bad[~nan], y[~nan]) and torch.equal(bad_r[~nan], rstd[~nan])
    dx, dw, db = timed_out(cuda_lib, 0, lambda: cuda_lib.norm_backward(dy, x, w, mean, rstd))
    nan = torch.isnan(dx).all(1)
    assert 0 < int(nan.sum()) < T and torch.equal(dx[~nan], want[0][~nan]) and torch.isnan(dw).all() and torch.isnan(db).all()
    assert torch.equal(cuda_lib.norm(x, w)[0], y)
    assert all(torch.equal(a, b) for a, b in zip(want, cuda_lib.norm_backward(dy, x, w, mean, rstd)))


@pytest.mark.parametrize("M,N,K", [(64, 512, 2048), (200, 256, 512), (3000, 2816, 512)])
def test_linear(cuda_lib, M, N, K):
    x, w, r = randn((M, K), 1, BF), randn((N, K), 2, BF, 0.05), randn((M, N), 3, BF)
    y = cuda_lib.linear(x, w, None, r, activation=1)
    bad = timed_out(cuda_lib, 2, lambda: cuda_lib.linear(x, w, None, r, activation=1))
    nan = torch.isnan(bad)
    assert 0 < int(nan.sum()) and torch.isnan(bad[0, 0]) and torch.equal(bad[~nan], y[~nan])
    assert M * N <= 256 * 256 or not nan.all()
    assert torch.equal(cuda_lib.linear(x, w, None, r, activation=1), y)
