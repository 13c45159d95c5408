"""The matrix product with its fused epilogue and its backward against plain
64-bit forms.

Tolerances.  A product of bf16 numbers is exact in fp32; a sum of K of them,
whatever its order, is off by at most 2 K e sum |a b| (e = 2^-24; the factor 2
allows truncating adders).  The activations' slopes are at most 1.13, and
expf / erff add a few e of |z|.  Then half an ulp of the output's type.  dz
is rounded to bf16 before its products (half an ulp of each dz) unless there is no
activation.
"""
import pytest
import torch

from _layers import EPS32 as E, HALF_ULP, act64, checkpoint64, randn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1, 1), (1, 4096, 2048), (2, 8, 64), (3, 250, 65), (17, 1000, 7), (64, 257, 1001), (128, 256, 64),
         (129, 640, 1024), (300, 130, 4096), (1000, 96, 520), (2500, 2600, 192)]


def laid_out(t, odd):
    """The tensor, or a view of it inside a wider buffer of NaN with rows off 16 bytes."""
    if not odd:
        return t
    buf = torch.full((t.shape[0], t.shape[1] + 7), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, 3:3 + t.shape[1]] = t
    return buf[:, 3:3 + t.shape[1]]


def close(got, want, bound, what):
    d = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    assert bool((d <= bound).all()), f"{what}: {(d - bound).max().item():.3g} over the bound, |d| {d.max().item():.3g}"


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("odd", [False, True])
def test_sums_are_exact_on_whole_numbers(cuda_lib, M, N, K, odd):
    """Small whole numbers: every partial sum is exact in any order, so a wrong
    index, a dropped or a doubled term shows as an inequality."""
    g = torch.Generator().manual_seed(M + N + K)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g).to(BF).cuda()
    x, w, r = ints(M, K), ints(N, K), ints(M, N)
    b = torch.randint(-9, 10, (N,), generator=g).float().cuda()
    y = cuda_lib.linear(laid_out(x, odd), laid_out(w, odd), b, laid_out(r, odd), out_dtype=F32)
    assert torch.equal(y.double(), x.double() @ w.double().t() + b.double() + r.double())
    dy = ints(M, N)
    dx, dw, db = cuda_lib.linear_backward(laid_out(dy, odd), laid_out(x, odd), laid_out(w, odd), grad_dtype=F32)
    assert torch.equal(dx.double(), dy.double() @ w.double())
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))
    ck = cuda_lib.checkpoint_pack(x)
    assert torch.equal(cuda_lib.linear_backward(dy, ck, w)[1], dw)      # |x| <= 4 is exact in 8 bits


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("bias,res,out,odd", [(F32, True, BF, False), (BF, False, F32, False), (None, True, F32, True),
                                              (F32, False, BF, True)])
def test_forward(cuda_lib, M, N, K, act, bias, res, out, odd):
    x, w = randn((M, K), 1, BF), randn((N, K), 2, BF, K ** -0.5)
    b = None if bias is None else randn((N,), 3, bias)
    r = randn((M, N), 4, BF) if res else None
    y, z = cuda_lib.linear(laid_out(x, odd), laid_out(w, odd), b, None if r is None else laid_out(r, odd),
                           activation=act, return_preact=True, out_dtype=out)
    zr = x.double() @ w.double().t() + (0 if b is None else b.double())
    dz = 2 * K * E * (x.double().abs() @ w.double().abs().t()) + 2 * E * zr.abs() + (0 if b is None else 2 * E * b.double().abs())
    close(z, zr, dz + HALF_ULP[BF] * (zr.abs() + dz), "z")
    yr = act64(zr, act)[0]
    dy = 1.13 * dz + 8 * E * (zr.abs() + 1)
    if r is not None:
        yr = yr + r.double()
        dy = dy + 2 * E * yr.abs() + E * r.double().abs()
    close(y, yr, dy + HALF_ULP[out] * (yr.abs() + dy), "y")
    only = cuda_lib.linear(laid_out(x, odd), laid_out(w, odd), b, r, activation=act, out_dtype=out)
    assert torch.equal(only, y)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("keep,wdt,odd", [(False, F32, False), (True, BF, False), (False, BF, True)])
def test_backward(cuda_lib, M, N, K, act, keep, wdt, odd):
    x, w = randn((M, K), 5, BF), randn((N, K), 6, BF, K ** -0.5)
    z, dy = randn((M, N), 7, BF, 1.5), randn((M, N), 8, BF, 0.1)
    kept = cuda_lib.checkpoint_pack(x) if keep else laid_out(x, odd)
    dx, dw, db = cuda_lib.linear_backward(laid_out(dy, odd), kept, laid_out(w, odd), laid_out(z, odd) if act else None,
                                          activation=act, grad_dtype=BF, weight_grad_dtype=wdt)
    xv = checkpoint64(x)[2].cuda() if keep else x.double()
    slope = act64(z, act)[1]
    g = dy.double() * slope
    fp = dy.double().abs() * 16 * E * (slope.abs() + z.double().abs() + 1) * bool(act)   # dz in fp32
    dg = fp + (HALF_ULP[BF] * (g.abs() + fp) if act else 0)                              # and as bf16
    ga = g.abs() + dg
    close(db, g.sum(0), (M + 8) * E * ga.sum(0) + fp.sum(0), "db")
    b1 = dg @ w.double().abs() + 2 * N * E * (ga @ w.double().abs())
    dxr = g @ w.double()
    close(dx, dxr, b1 + HALF_ULP[BF] * (dxr.abs() + b1), "dx")
    b2 = dg.t() @ xv.abs() + 2 * M * E * (ga.t() @ xv.abs())
    dwr = g.t() @ xv
    close(dw, dwr, b2 + HALF_ULP[wdt] * (dwr.abs() + b2), "dw")


def test_gradient_against_differences(cuda_lib):
    M, N, K = 12, 40, 24
    x, w, b = randn((M, K), 11, BF), randn((N, K), 12, BF, 0.2), randn((N,), 13)
    dy = randn((M, N), 14, BF)
    for act in (1, 2):
        _, z = cuda_lib.linear(x, w, b, activation=act, return_preact=True)
        # z is kept in bf16: the formula is differentiated at that z, so move it there by the bias
        shift = z.double() - (x.double() @ w.double().t() + b.double())
        grads = cuda_lib.linear_backward(dy, x, w, z, activation=act, grad_dtype=F32)
        for i, g in enumerate(grads):
            ps = [x.double(), w.double(), b.double()]
            v = randn(tuple(ps[i].shape), 30 + i).double()
            ends = []
            for s in (1e-5, -1e-5):
                q = list(ps)
                q[i] = q[i] + s * v
                ends.append((dy.double() * act64(q[0] @ q[1].t() + q[2] + shift, act)[0]).sum())
            want, got = (ends[0] - ends[1]) / 2e-5, (g.double() * v).sum()
            # dz as bf16: half an ulp of every term
            assert abs(got - want) <= (1e-6 if i == 2 else 2.0 ** -8) * (g.double() * v).abs().sum() + 1e-6


def test_accumulate_and_chosen_gradients(cuda_lib):
    M, N, K = 70, 96, 136
    x, w, dy, z = randn((M, K), 1, BF), randn((N, K), 2, BF), randn((M, N), 3, BF), randn((M, N), 4, BF)
    dx, dw, db = cuda_lib.linear_backward(dy, x, w, z, activation=1)
    aw, ab = torch.ones(N, K, device="cuda"), torch.ones(N, device="cuda")
    cuda_lib.linear_backward(dy, x, w, z, activation=1, grad_weight=aw, grad_bias=ab, accumulate=True)
    assert torch.equal(aw, dw + 1) and torch.equal(ab, db + 1)
    with pytest.raises(cuda_lib.RlkError):
        cuda_lib.linear_backward(dy, x, w, z, activation=1, grad_weight=aw.to(BF), grad_bias=ab, accumulate=True)
    for wx, ww, wb in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)):
        got = cuda_lib.linear_backward(dy, x, w, z, activation=1, want_x_grad=wx, want_weight_grad=ww, want_bias_grad=wb)
        for t, on, full in zip(got, (wx, ww, wb), (dx, dw, db)):
            assert (t is None and not on) or torch.equal(t, full)


def test_no_rows(cuda_lib):
    x, w = torch.empty((0, 64), dtype=BF, device="cuda"), randn((32, 64), 1, BF)
    assert cuda_lib.linear(x, w).shape == (0, 32)
    dx, dw, db = cuda_lib.linear_backward(torch.empty((0, 32), dtype=BF, device="cuda"), x, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
    aw, ab = torch.ones(32, 64, device="cuda"), torch.ones(32, device="cuda")
    cuda_lib.linear_backward(torch.empty((0, 32), dtype=BF, device="cuda"), x, w, grad_weight=aw, grad_bias=ab, accumulate=True)
    assert bool((aw == 1).all()) and bool((ab == 1).all())


@pytest.mark.parametrize("M", [5, 300])
def test_residual_in_place_and_nothing_outside(cuda_lib, M):
    N, K = 300, 128
    x, w, r = randn((M, K), 1, BF), randn((N, K), 2, BF, 0.1), randn((M, N), 3, BF)
    want = cuda_lib.linear(x, w, None, r, activation=2)
    buf = torch.full((M + 2, N + 12), 123.0, dtype=BF, device="cuda")
    inner = buf[1:M + 1, 4:4 + N]
    inner.copy_(r)
    cuda_lib.linear(x, w, None, inner, activation=2, out=inner)
    assert torch.equal(inner, want)
    inner.fill_(123.0)
    assert bool((buf == 123.0).all())


@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (200, 256, 512)])
def test_bad_values_stay_in_their_rows(cuda_lib, M, N, K):
    x, w = randn((M, K), 1, BF), randn((N, K), 2, BF, 0.1)
    good = cuda_lib.linear(x, w)
    x2 = x.clone()
    x2[0, K - 1] = float("nan")
    got = cuda_lib.linear(x2, w)
    assert torch.isnan(got[0]).all() and torch.equal(got[1:], good[1:])
    x2[0] = 0
    w2 = w.clone()
    w2[3, 5] = float("inf")
    got = cuda_lib.linear(x2, w2)
    assert torch.isnan(got[0, 3]) and torch.isfinite(got[0, :3]).all() and torch.isfinite(got[:, 4:]).all()


def test_repeats_streams_and_graphs(cuda_lib):
    for M, N, K in ((1, 1024, 4096), (600, 1030, 1001)):
        x, w, b, r = randn((M, K), 1, BF), randn((N, K), 2, BF, 0.05), randn((N,), 3), randn((M, N), 4, BF)
        dy = randn((M, N), 5, BF)

        def step():
            y, z = cuda_lib.linear(x, w, b, r, activation=1, return_preact=True)
            return (y, z) + cuda_lib.linear_backward(dy, x, w, z, activation=1)
        want = step()
        assert all(torch.equal(a, c) for a, c in zip(want, step()))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = step()
        s.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_autograd_matches_the_calls(cuda_lib):
    x, w, b, r = randn((20, 96), 1, BF), randn((64, 96), 2, BF), randn((64,), 3), randn((20, 64), 4, BF)
    dy = randn((20, 64), 5, BF)
    for act in (0, 1):
        for keep in (False, True):
            ps = [t.clone().requires_grad_() for t in (x, w, b, r)]
            cuda_lib.linear_autograd(*ps, activation=act, keep_8bit=keep).backward(dy)
            _, z = cuda_lib.linear(x, w, b, r, activation=act, return_preact=True)
            kept = cuda_lib.checkpoint_pack(x) if keep else x
            dx, dw, db = cuda_lib.linear_backward(dy, kept, w, z, activation=act, weight_grad_dtype=BF)
            assert all(torch.equal(p.grad, q) for p, q in zip(ps, (dx, dw, db, dy)))


@pytest.mark.parametrize("M,N,K", [(2601, 2003, 4100), (4100, 2601, 2003), (2600, 2560, 4096)])
def test_many_rounds_of_tiles(cuda_lib, M, N, K):
    """More tiles of 256 x 256 than pairs of SMs, a ragged last round and a long K
    (forward; and dw, whose K is M).  Small whole numbers, so every sum is exact."""
    g = torch.Generator().manual_seed(M)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).to(BF).cuda()
    x, w, r, dy = ints(M, K), ints(N, K), ints(M, N), ints(M, N)
    for _ in range(2):
        y = cuda_lib.linear(x, w, None, r, out_dtype=F32)
        dx, dw, db = cuda_lib.linear_backward(dy, x, w, grad_dtype=F32)
        assert torch.equal(y, x.float() @ w.float().t() + r.float())
        assert torch.equal(dx, dy.float() @ w.float()) and torch.equal(dw, dy.float().t() @ x.float())
        assert torch.equal(db, dy.float().sum(0))


@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K,pad", [(2560, 7490, 0), (300, 65, 1), (300, 66, 0), (300, 66, 1), (7, 1, 1), (5000, 4098, 0)])
def test_few_rows_of_any_alignment(cuda_lib, M, N, K, pad):
    """Rows on 4-byte and on 2-byte boundaries; whole numbers, so the sums are exact."""
    x, w = (torch.full((r, K + pad), float("nan"), device="cuda", dtype=BF)[:, :K] for r in (M, N))
    x.copy_((torch.arange(M * K, device="cuda") % 13 - 6).view(M, K))
    w.copy_((torch.arange(N * K, device="cuda") * 7 % 11 - 5).view(N, K))
    y = cuda_lib.linear(x, w, out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w.double().T)
