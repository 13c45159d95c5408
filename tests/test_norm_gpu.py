"""Layer / RMS norm and the 8-bit activation checkpoints against plain 64-bit
forms.

Tolerances.  A sum of H terms whose longest chain of additions is n has an
error of at most n 2^-24 times the sum of the terms' magnitudes.  The kernels
give each thread at most H / 32 terms (few rows' threads are a warp) and join
at most 16 + 5 partial sums, so with n = H / 32 + 32 (capped at H + 8)
  |mean - m| <= n e mean|x|,   |rstd - r| <= r (n + 8) e,
and each output's bound follows by propagating these through its formula, plus
half an ulp of its type.  Parameter gradients add T terms: chains of at most
T / parts + parts + 8, which T + 16 bounds.
"""
import pytest
import torch

from _layers import EPS32, HALF_ULP, checkpoint64, norm64, norm_grad64, randn, rows

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (1, 4096), (2, 7), (3, 31), (5, 32), (4, 33), (7, 1003), (130, 4096), (37, 5003),
          (1000, 64), (9, 8192), (6, 8200), (5, 16384), (3, 40001)]


def steps(H):
    return min(H + 8, H / 32 + 32)


def close(got, want, bound, what):
    d = (got.double() - want).abs()
    worst = (d - bound).max().item()
    assert torch.isfinite(got).all() and worst <= 0, f"{what}: {worst:.3g} over the bound, |d| {d.max().item():.3g}"


def params(H, seed, has_w, has_b, dtype):
    w = (1.0 + 0.1 * randn((H,), seed)).to(dtype) if has_w else None
    b = randn((H,), seed + 1, scale=0.1).to(dtype) if has_b else None
    return w, b


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("rms", [0, 1])
@pytest.mark.parametrize("dtype,pdtype,odd", [(BF, F32, False), (F32, BF, False), (BF, BF, True), (F32, F32, True)])
def test_forward(cuda_lib, T, H, rms, dtype, pdtype, odd):
    x = rows(T, H, dtype, 1, odd_layout=odd)
    w, b = params(H, 2, H != 7, not rms, pdtype)
    y, mean, rstd = cuda_lib.norm(x, w, b, kind=rms, eps=1e-5)
    yr, m, r = norm64(x, w, b, rms, 1e-5)
    e, n = EPS32, steps(H)
    dm = (n + 4) * e * x.double().abs().mean(1)
    if not rms:
        close(mean, m, dm, "mean")
        # the mean's own error moves the variance only in second order
        dr = r * ((n + 8) * e + 0.5 * (dm * r).square())
    else:
        assert mean is None
        dr = r * (n + 8) * e
    close(rstd, r, dr, "rstd")
    W = torch.ones(H, device="cuda").double() if w is None else w.double()
    h = (x.double() - m[:, None]) * r[:, None]
    bound = W.abs() * (r[:, None] * ((0 if rms else dm)[:, None] if not rms else 0)
                       + h.abs() * ((dr / r)[:, None] + 4 * e)) + 2 * e * yr.abs() + HALF_ULP[dtype] * yr.abs() * (1 + 2.0 ** -6) + 1e-38
    assert y.dtype == dtype
    close(y, yr, bound, "y")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("rms", [0, 1])
@pytest.mark.parametrize("dtype,dyt,keep,odd", [(BF, F32, False, False), (BF, BF, True, False), (F32, F32, True, False),
                                                (BF, BF, False, True), (F32, BF, False, False)])
def test_backward(cuda_lib, T, H, rms, dtype, dyt, keep, odd):
    x = rows(T, H, dtype, 3, odd_layout=odd)
    w, b = params(H, 4, H != 7, not rms, F32)
    dy = randn((T, H), 5, scale=0.01, dtype=dyt)
    ck = cuda_lib.new_checkpoint(T, H, "cuda") if keep else None
    y, mean, rstd = cuda_lib.norm(x, w, b, kind=rms, checkpoint=ck)
    dx, dw, db = cuda_lib.norm_backward(dy, ck if keep else x, w, mean, rstd, kind=rms, grad_dtype=dtype)
    xv = checkpoint64(x)[2].cuda() if keep else x.double()
    m64 = torch.zeros(T, device="cuda", dtype=torch.float64) if rms else mean.double()
    dxr, dwr, dbr = norm_grad64(dy, xv, w, m64, rstd, rms)
    # the statistics are the kernel's own, so what is left is the formula's rounding
    e, n = EPS32, steps(H)
    h = (xv - m64[:, None]) * rstd.double()[:, None]
    g = dy.double() if w is None else dy.double() * w.double()
    mag = g.abs() + h.abs() * (g * h).abs().mean(1, keepdim=True) + g.abs().mean(1, keepdim=True)
    hx = 4 * e * (h.abs() + rstd.double()[:, None] * xv.abs())
    bound = rstd.double()[:, None].abs() * ((n + 12) * e * mag + 2 * hx * (g * h).abs().mean(1, keepdim=True)
                                            + h.abs() * (g.abs() * hx).mean(1, keepdim=True))
    close(dx, dxr, bound + HALF_ULP[dtype] * dxr.abs() * (1 + 2.0 ** -6) + 1e-38, "dx")
    close(dw, dwr, (T + 16) * e * (dy.double() * h).abs().sum(0) + (dy.double().abs() * hx).sum(0), "dw")
    close(db, dbr, (T + 16) * e * dy.double().abs().sum(0), "db")


@pytest.mark.parametrize("rms", [0, 1])
def test_gradients_against_differences(cuda_lib, rms):
    """<dL/dp, v> for p = x, weight, bias against central differences of the
    64-bit forward along v (error: step^2 times third derivatives, ~1e-8, and the
    kernel's fp32)."""
    T, H = 6, 320
    x, (w, b) = rows(T, H, F32, 7), params(H, 8, True, True, F32)
    dy = randn((T, H), 9)
    y, mean, rstd = cuda_lib.norm(x, w, b, kind=rms)
    grads = cuda_lib.norm_backward(dy, x, w, mean, rstd, kind=rms)
    for i, g in enumerate(grads):
        ps = [x.double(), w.double(), b.double()]
        v = randn(tuple(ps[i].shape), 20 + i).double()
        ends = []
        for s in (1e-5, -1e-5):
            q = list(ps)
            q[i] = q[i] + s * v
            ends.append((dy.double() * norm64(q[0], q[1], q[2], rms, 1e-5)[0]).sum())
        want = (ends[0] - ends[1]) / 2e-5
        got = (g.double() * v).sum()
        assert abs(got - want) <= 1e-5 * (g.double() * v).abs().sum() + 1e-7


def test_accumulate_and_partial_outputs(cuda_lib):
    T, H = 33, 96
    x, dy = rows(T, H, BF, 1), randn((T, H), 2)
    w, b = params(H, 3, True, True, F32)
    y, mean, rstd = cuda_lib.norm(x, w, b)
    dx, dw, db = cuda_lib.norm_backward(dy, x, w, mean, rstd)
    aw, ab = torch.ones(H, device="cuda"), torch.full((H,), 2.0, device="cuda")
    cuda_lib.norm_backward(dy, x, w, mean, rstd, grad_weight=aw, grad_bias=ab, accumulate=True)
    assert torch.equal(aw, dw + 1.0) and torch.equal(ab, db + 2.0)
    d2, w2, b2 = cuda_lib.norm_backward(dy, x, w, mean, rstd, want_bias_grad=False)
    assert torch.equal(d2, dx) and torch.equal(w2, dw) and b2 is None
    d3, w3, b3 = cuda_lib.norm_backward(dy, x, w, mean, rstd, want_weight_grad=False, want_bias_grad=False)
    assert torch.equal(d3, dx) and w3 is None and b3 is None


def test_no_rows(cuda_lib):
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    y, mean, rstd = cuda_lib.norm(x)
    assert y.shape == (0, 64) and rstd.numel() == 0
    dx, dw, db = cuda_lib.norm_backward(x, x, None, mean, rstd)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("H", [96, 4096, 5003])
def test_bad_rows_stay_alone(cuda_lib, H):
    """A NaN, an infinity and an overflowing row give NaN rows and the status
    bit; the other rows keep their bits."""
    x = rows(8, H, F32, 11)
    good = cuda_lib.norm(x)[0]
    bad = x.clone()
    bad[1, H // 2], bad[3, 0], bad[5, H - 1] = float("nan"), float("inf"), 1e30
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ck = cuda_lib.new_checkpoint(8, H, "cuda")
    y, mean, rstd = cuda_lib.norm(bad, status_word=st, checkpoint=ck)
    for t in range(8):
        if t in (1, 3, 5):
            assert torch.isnan(y[t]).all() and torch.isnan(rstd[t]) and torch.isnan(mean[t])
        else:
            assert torch.equal(y[t], good[t])
    assert int(st) == cuda_lib.STATUS_NONFINITE
    dx, dw, db = cuda_lib.norm_backward(torch.ones_like(x), ck, None, mean, rstd)
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[0]).all() and torch.isnan(dw).all()


@pytest.mark.parametrize("H", [64, 1003, 4096, 20000])
def test_rows_do_not_depend_on_the_batch(cuda_lib, H):
    x, w = rows(50, H, BF, 13), randn((H,), 14)
    y, mean, rstd = cuda_lib.norm(x, w)
    for lo, hi in ((0, 1), (17, 50)):
        y2, m2, r2 = cuda_lib.norm(x[lo:hi].clone(), w)
        assert torch.equal(y2, y[lo:hi]) and torch.equal(m2, mean[lo:hi]) and torch.equal(r2, rstd[lo:hi])


def test_runs_repeat_bit_for_bit(cuda_lib):
    x, w, dy = rows(700, 4096, BF, 15), randn((4096,), 16), randn((700, 4096), 17)
    y, m, r = cuda_lib.norm(x, w)
    first = cuda_lib.norm_backward(dy, x, w, m, r)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, cuda_lib.norm_backward(dy, x, w, m, r)))


def test_autograd_matches_the_calls(cuda_lib):
    x, w, b = rows(12, 256, BF, 18), randn((256,), 19), randn((256,), 20)
    dy = randn((12, 256), 21, dtype=BF)
    for keep in (False, True):
        xs, ws, bs = x.clone().requires_grad_(), w.clone().requires_grad_(), b.clone().requires_grad_()
        y = cuda_lib.norm_autograd(xs, ws, bs, keep_8bit=keep)
        y.backward(dy)
        ck = cuda_lib.new_checkpoint(12, 256, "cuda")
        y2, m, r = cuda_lib.norm(x, w, b, checkpoint=ck)
        dx, dw, db = cuda_lib.norm_backward(dy, ck if keep else x, w, m, r, grad_dtype=BF)
        assert torch.equal(y, y2) and torch.equal(xs.grad, dx) and torch.equal(ws.grad, dw) and torch.equal(bs.grad, db)


# ------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("T,H", [(1, 1), (3, 31), (2, 32), (4, 33), (5, 48), (7, 1003), (64, 4096), (3, 16384), (300, 40)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("odd", [False, True])
def test_checkpoint_is_exact(cuda_lib, T, H, dtype, odd):
    """Codes, scales and values equal the definition's (every step but one
    rounding is exact, so there is no tolerance)."""
    x = rows(T, H, dtype, 31, odd_layout=odd)
    ck = cuda_lib.checkpoint_pack(x)
    codes, scales, vals = checkpoint64(x)
    assert torch.equal(ck.codes[:, :H].cpu(), codes) and torch.equal(ck.scales[:, :scales.shape[1]].cpu(), scales)
    for out in (BF, F32):
        assert torch.equal(cuda_lib.checkpoint_unpack(ck, dtype=out).double().cpu(), vals)
    nb = -(-H // 32)
    top = torch.nn.functional.pad(x.double().abs().cpu(), (0, nb * 32 - H)).view(T, nb, 32).amax(2)
    err = torch.nn.functional.pad((vals - x.double().cpu()).abs(), (0, nb * 32 - H)).view(T, nb, 32).amax(2)
    assert bool((err <= top / 127 * (1 + 1e-12)).all())


def test_checkpoint_edges(cuda_lib):
    """Blocks of zeros, subnormals, the largest numbers, step boundaries, ties,
    NaN and infinities."""
    x = torch.zeros((1, 32 * 10), device="cuda")
    x[0, 32:64] = 1e-44
    x[0, 64:96] = torch.finfo(torch.float32).max
    x[0, 96] = 127.0
    x[0, 97:100] = torch.tensor([0.5, 1.5, -2.5])          # ties at step 1
    x[0, 128] = 127.00001
    x[0, 160] = 63.5
    x[0, 192] = float("nan")
    x[0, 224], x[0, 225] = -float("inf"), 3.0
    x[0, 256] = 127 * 2.0 ** -126
    x[0, 288] = -1e-3
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ck = cuda_lib.checkpoint_pack(x, status_word=st)
    codes, scales, vals = checkpoint64(x)
    assert torch.equal(ck.codes[:, :320].cpu(), codes) and torch.equal(ck.scales[:, :10].cpu(), scales)
    got = cuda_lib.checkpoint_unpack(ck, dtype=F32).double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(vals)) and torch.equal(got.nan_to_num(7.0), vals.nan_to_num(7.0))
    assert int(st) == cuda_lib.STATUS_NONFINITE and scales[0].tolist()[6:8] == [255, 255]
    assert codes[0, 97:100].tolist() == [0, 2, -2] and scales[0, 3] == 127 and scales[0, 4] == 128


@pytest.mark.parametrize("H", [64, 1003, 4096, 9000])
def test_norm_writes_the_same_checkpoint(cuda_lib, H):
    x = rows(9, H, BF, 33)
    ck = cuda_lib.new_checkpoint(9, H, "cuda")
    cuda_lib.norm(x, checkpoint=ck)
    alone = cuda_lib.checkpoint_pack(x)
    nb = -(-H // 32)
    assert torch.equal(ck.codes[:, :H], alone.codes[:, :H]) and torch.equal(ck.scales[:, :nb], alone.scales[:, :nb])


def test_nothing_is_written_outside(cuda_lib):
    """Outputs inside larger buffers: what lies around them stays."""
    T, H = 7, 1003
    x, dy = rows(T, H, BF, 35), randn((T, H), 36)
    mark = 123.0
    ybuf = torch.full((T + 2, H + 9), mark, device="cuda", dtype=BF)
    cuda_lib.norm(x, out=ybuf[1:T + 1, 4:4 + H])
    _, m, r = cuda_lib.norm(x)
    gbuf = torch.full((T + 2, H + 9), mark, device="cuda")
    cuda_lib.norm_backward(dy, x, None, m, r, out=gbuf[1:T + 1, 4:4 + H])
    for buf in (ybuf, gbuf):
        inner = buf[1:T + 1, 4:4 + H].clone()
        buf[1:T + 1, 4:4 + H] = mark
        assert bool((buf == mark).all()) and torch.isfinite(inner).all()
    codes = torch.full((T + 2, 1024), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((T + 2, 48), 77, dtype=torch.uint8, device="cuda")
    cuda_lib.checkpoint_pack(x, out=cuda_lib.Checkpoint(codes[1:T + 1], scales[1:T + 1], T, H))
    assert bool((codes[0] == 77).all()) and bool((codes[T + 1] == 77).all()) and bool((codes[:, H:] == 77).all())
    assert bool((scales[0] == 77).all()) and bool((scales[T + 1] == 77).all()) and bool((scales[:, 32:] == 77).all())


def test_another_stream(cuda_lib):
    x, dy, w = rows(64, 512, BF, 37), randn((64, 512), 38), randn((512,), 39)
    y, m, r = cuda_lib.norm(x, w)
    want = cuda_lib.norm_backward(dy, x, w, m, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, m2, r2 = cuda_lib.norm(x, w)
        got = cuda_lib.norm_backward(dy, x, w, m2, r2)
    s.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(want, got))
