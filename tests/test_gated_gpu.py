"""The gated linear layer and its backward against plain 64-bit forms.

Tolerances as for the linear layer: a sum of K products of bf16 numbers is off by at
most 2 K e sum |a b| (e = 2^-24), act and its slope by a few e of their arguments, a
slope is at most 1.13 and |act(z)| <= |z|; then half an ulp of the output's type.  dg and
du are rounded to bf16 (half an ulp each) before their products.
"""
import pytest
import torch

from _distil import act64
from _layers import EPS32 as E, HALF_ULP, checkpoint64, randn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1, 1), (1, 2048, 4096), (2, 8, 64), (3, 250, 65), (4, 130, 1000), (5, 70, 200), (17, 1000, 7), (64, 257, 1001), (128, 256, 64),
         (129, 640, 1024), (300, 130, 4096), (520, 1301, 1003), (1000, 96, 520), (2500, 1400, 192)]


def laid_out(t, odd):
    """The tensor, or a view of it inside a wider buffer of NaN with rows off 16 bytes (even: on 4)."""
    if not odd:
        return t
    lead = 2 if odd == "even" else 3
    buf = torch.full((t.shape[0], t.shape[1] + 7 + (t.shape[1] + 7) % 2 * (odd == "even")), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, lead:lead + t.shape[1]] = t
    return buf[:, lead:lead + t.shape[1]]


def close(got, want, bound, what):
    d = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    assert bool((d <= bound).all()), f"{what}: {(d - bound).max().item():.3g} over the bound, |d| {d.max().item():.3g}"


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("odd", [False, True, "even"])
def test_sums_are_exact_on_whole_numbers(cuda_lib, M, N, K, odd):
    """Small whole numbers without an activation: every partial sum is exact in any order, so a
    wrong index, a dropped or a doubled term, gate taken for up, shows as an inequality."""
    rlk = cuda_lib
    g = torch.Generator().manual_seed(M + N + K)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g).to(BF).cuda()
    x, wg, wu = ints(M, K), ints(N, K), ints(N, K)
    K3 = K if K <= 520 else 520                       # |g| <= 9 K: the product of two stays exact below 2^24
    wg[:, K3:] = 0
    x, wg, wu = (t.sign() if K > 200 else t for t in (x, wg, wu))
    bg, bu = (torch.randint(-9, 10, (N,), generator=g).float().cuda() for _ in range(2))
    gr, ur = x.double() @ wg.double().t() + bg.double(), x.double() @ wu.double().t() + bu.double()
    assert (gr * ur).abs().max() < 2 ** 24
    y = rlk.gated_linear(laid_out(x, odd), laid_out(wg, odd), laid_out(wu, odd), bg, bu, activation=rlk.ACT_NONE, out_dtype=F32)
    assert torch.equal(y.double(), gr * ur)
    dy, gate, up = ints(M, N), ints(M, N), ints(M, N)
    dx, dwg, dwu, dbg, dbu = rlk.gated_linear_backward(laid_out(dy, odd), laid_out(x, odd), laid_out(wg, odd), laid_out(wu, odd), laid_out(gate, odd),
                                                       laid_out(up, odd), activation=rlk.ACT_NONE, grad_dtype=F32)
    dg, du = dy.double() * up.double(), dy.double() * gate.double()
    assert torch.equal(dx.double(), dg @ wg.double() + du @ wu.double())
    assert torch.equal(dwg.double(), dg.t() @ x.double()) and torch.equal(dwu.double(), du.t() @ x.double())
    assert torch.equal(dbg.double(), dg.sum(0)) and torch.equal(dbu.double(), du.sum(0))
    got = rlk.gated_linear_backward(dy, rlk.checkpoint_pack(x), wg, wu, gate, up, activation=rlk.ACT_NONE, want_x_grad=False)
    assert got[0] is None and torch.equal(got[1], dwg) and torch.equal(got[2], dwu)      # |x| <= 4 is exact in 8 bits


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("bias,out,odd", [(F32, BF, False), (None, F32, False), (BF, F32, True), (F32, BF, True), (None, BF, "even")])
def test_forward(cuda_lib, M, N, K, act, bias, out, odd):
    rlk = cuda_lib
    x, wg, wu = randn((M, K), 1, BF), randn((N, K), 2, BF, K ** -0.5), randn((N, K), 3, BF, K ** -0.5)
    bg, bu = (None, None) if bias is None else (randn((N,), 4, bias), randn((N,), 5, bias))
    y, g, u = rlk.gated_linear(laid_out(x, odd), laid_out(wg, odd), laid_out(wu, odd), bg, bu, activation=act, return_preact=True, out_dtype=out)
    want, off = [], []
    for w, b in ((wg, bg), (wu, bu)):
        z = x.double() @ w.double().t() + (0 if b is None else b.double())
        want.append(z)
        off.append(2 * K * E * (x.double().abs() @ w.double().abs().t()) + 2 * E * z.abs() + (0 if b is None else 2 * E * b.double().abs()))
    for got, z, d, name in zip((g, u), want, off, ("gate", "up")):
        close(got, z, d + HALF_ULP[BF] * (z.abs() + d), name)
    a = act64(want[0], act)[0]
    da = 1.13 * off[0] + 8 * E * (a.abs() + 1)
    yr = a * want[1]
    dy = da * want[1].abs() + (a.abs() + da) * off[1] + 2 * E * yr.abs()
    close(y, yr, dy + HALF_ULP[out] * (yr.abs() + dy), "y")
    room = torch.full((M, N + 5), 7.0, dtype=out, device="cuda")
    only = rlk.gated_linear(laid_out(x, odd), laid_out(wg, odd), laid_out(wu, odd), bg, bu, activation=act, out=room[:, 2:2 + N])
    assert torch.equal(only, y) and (room[:, :2] == 7).all() and (room[:, 2 + N:] == 7).all()


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("keep,wdt,odd", [(False, F32, False), (True, BF, False), (False, BF, True)])
def test_backward(cuda_lib, M, N, K, act, keep, wdt, odd):
    rlk = cuda_lib
    x, wg, wu = randn((M, K), 5, BF), randn((N, K), 6, BF, K ** -0.5), randn((N, K), 7, BF, K ** -0.5)
    gate, up, dy = randn((M, N), 8, BF, 1.5), randn((M, N), 9, BF), randn((M, N), 10, BF, 0.1)
    kept = rlk.checkpoint_pack(x) if keep else laid_out(x, odd)
    dx, dwg, dwu, dbg, dbu = rlk.gated_linear_backward(laid_out(dy, odd), kept, laid_out(wg, odd), laid_out(wu, odd), laid_out(gate, odd), laid_out(up, odd),
                                                       activation=act, weight_grad_dtype=wdt)
    xv = checkpoint64(x)[2].cuda() if keep else x.double()
    value, slope = act64(gate, act)
    z = gate.double().abs()
    g, u = dy.double() * up.double() * slope, dy.double() * value
    fg = dy.double().abs() * up.double().abs() * 16 * E * (slope.abs() + z + 1)          # in fp32
    fu = dy.double().abs() * 16 * E * (value.abs() + z + 1)
    dxr, bound = 0, 0
    for d, f, w, dw, db, name in ((g, fg, wg, dwg, dbg, "gate"), (u, fu, wu, dwu, dbu, "up")):
        off = f + HALF_ULP[BF] * (d.abs() + f)                                           # and as bf16
        most = d.abs() + off
        close(db, d.sum(0), (M + 8) * E * most.sum(0) + f.sum(0), "bias of " + name)
        b2 = off.t() @ xv.abs() + 2 * M * E * (most.t() @ xv.abs())
        want = d.t() @ xv
        close(dw, want, b2 + HALF_ULP[wdt] * (want.abs() + b2), "weight of " + name)
        dxr = dxr + d @ w.double()
        bound = bound + off @ w.double().abs() + 4 * N * E * (most @ w.double().abs())
    close(dx, dxr, bound + HALF_ULP[BF] * (dxr.abs() + bound), "dx")


def test_gradients_against_differences(cuda_lib):
    """The gradients against central differences of the 64-bit forward, at the kept projections."""
    rlk, M, N, K = cuda_lib, 12, 40, 24
    x, wg, wu, dy = randn((M, K), 11, BF), randn((N, K), 12, BF, 0.2), randn((N, K), 13, BF, 0.2), randn((M, N), 14, BF)
    bg, bu = randn((N,), 15), randn((N,), 16)
    for act in (0, 1, 2):
        _, gate, up = rlk.gated_linear(x, wg, wu, bg, bu, activation=act, return_preact=True)
        # the projections are kept in bf16: the formula is differentiated there, moved by the biases
        shift = [z.double() - (x.double() @ w.double().t() + b.double()) for z, w, b in ((gate, wg, bg), (up, wu, bu))]
        grads = rlk.gated_linear_backward(dy, x, wg, wu, gate, up, activation=act, grad_dtype=F32)
        base = [t.double() for t in (x, wg, wu, bg, bu)]

        def loss(p):
            a = act64(p[0] @ p[1].t() + p[3] + shift[0], act)[0]
            return (dy.double() * a * (p[0] @ p[2].t() + p[4] + shift[1])).sum()

        for i, grad in enumerate(grads):
            v = randn(tuple(base[i].shape), 30 + i).double()
            ends = []
            for s in (1e-5, -1e-5):
                p = list(base)
                p[i] = p[i] + s * v
                ends.append(loss(p))
            slope = ((ends[0] - ends[1]) / 2e-5).item()
            got = (grad.double() * v).sum().item()
            # each of the terms is off by the bf16 rounding of dg or du, 2^-9 of it at most (root mean square a third)
            assert abs(got - slope) <= 2 ** -8 * (grad.double().abs() * v.abs()).sum().item() + 1e-6 * abs(slope)


def test_autograd_and_checkpoint(cuda_lib):
    rlk = cuda_lib
    x, wg, wu = (t.requires_grad_() for t in (randn((70, 96), 1, BF), randn((130, 96), 2, BF, 0.1), randn((130, 96), 3, BF, 0.1)))
    bg, bu = randn((130,), 4).requires_grad_(), randn((130,), 5).requires_grad_()
    dy = randn((70, 130), 6, BF)
    _, gate, up = rlk.gated_linear(x.detach(), wg.detach(), wu.detach(), bg.detach(), bu.detach(), return_preact=True)
    for keep in (False, True):
        rlk.gated_linear_autograd(x, wg, wu, bg, bu, keep_8bit=keep).backward(dy)
        kept = rlk.checkpoint_pack(x.detach()) if keep else x.detach()
        want = rlk.gated_linear_backward(dy, kept, wg.detach(), wu.detach(), gate, up, weight_grad_dtype=BF)
        for t, w in zip((x, wg, wu, bg, bu), want):
            assert torch.equal(t.grad, w)
            t.grad = None
    y = rlk.gated_linear_autograd(x.detach(), wg, wu.detach())
    y.backward(dy)
    assert wg.grad is not None and x.grad is None and wu.grad is None
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(rlk.gated_linear_autograd(x, wg, wu).float().sum(), x, create_graph=True)[0].float().sum(), x)


def test_accumulate_and_what_is_not_wanted(cuda_lib):
    rlk = cuda_lib
    x, wg, wu = randn((33, 40), 1, BF), randn((24, 40), 2, BF), randn((24, 40), 3, BF)
    gate, up, dy = randn((33, 24), 4, BF), randn((33, 24), 5, BF), randn((33, 24), 6, BF)
    dx, dwg, dwu, dbg, dbu = rlk.gated_linear_backward(dy, x, wg, wu, gate, up)
    to = [t.clone() for t in (dwg, dwu, dbg, dbu)]
    rlk.gated_linear_backward(dy, x, wg, wu, gate, up, want_x_grad=False, grad_w_gate=to[0], grad_w_up=to[1], grad_bias_gate=to[2], grad_bias_up=to[3],
                              accumulate=True)
    assert all(torch.equal(a, b + b) for a, b in zip(to, (dwg, dwu, dbg, dbu)))
    got = rlk.gated_linear_backward(dy, None, wg, wu, gate, up, want_weight_grad=False, want_bias_grad=False)
    assert torch.equal(got[0], dx) and got[1:] == (None,) * 4
    got = rlk.gated_linear_backward(dy, None, wg, wu, gate, up, want_x_grad=False, want_weight_grad=False)
    assert torch.equal(got[3], dbg) and torch.equal(got[4], dbu) and got[:3] == (None,) * 3
    wide = torch.full((2, 24, 50), 3.0, device="cuda")                # rows of a wider buffer
    got = rlk.gated_linear_backward(dy, x, wg, wu, gate, up, grad_w_gate=wide[0, :, 5:45], grad_w_up=wide[1, :, 5:45])
    assert torch.equal(got[1], dwg) and torch.equal(got[2], dwu) and (wide[:, :, :5] == 3).all() and (wide[:, :, 45:] == 3).all()
    # the halves of one matrix of weights
    both = torch.cat([wg, wu])
    assert torch.equal(rlk.gated_linear(x, both[:24], both[24:]), rlk.gated_linear(x, wg, wu))


def test_no_rows(cuda_lib):
    rlk = cuda_lib
    x, w = torch.empty(0, 40, dtype=BF, device="cuda"), randn((24, 40), 2, BF)
    z = torch.empty(0, 24, dtype=BF, device="cuda")
    assert rlk.gated_linear(x, w, w).shape == (0, 24)
    got = rlk.gated_linear_backward(z, x, w, w, z, z)
    assert got[0].shape == (0, 40) and all((t == 0).all() for t in got[1:])


def test_infinities_and_nan(cuda_lib):
    rlk = cuda_lib
    for M in (2, 40):
        x, wg, wu = randn((M, 64), 1, BF), randn((32, 64), 2, BF), randn((32, 64), 3, BF)
        want = rlk.gated_linear(x, wg, wu)
        x[1, 5] = float("nan")
        y = rlk.gated_linear(x, wg, wu)
        assert torch.isnan(y[1]).all() and torch.equal(y[0], want[0]) and torch.equal(y[2:], want[2:])


def test_streams_graph_and_repeat(cuda_lib):
    rlk = cuda_lib
    x, wg, wu = randn((200, 501), 1, BF), randn((301, 501), 2, BF, 0.05), randn((301, 501), 3, BF, 0.05)   # with copies of all three
    dy = randn((200, 301), 4, BF)

    def run():
        y, g, u = rlk.gated_linear(x, wg, wu, return_preact=True)
        return (y, g, u, *rlk.gated_linear_backward(dy, x, wg, wu, g, u))

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    x.copy_(randn((200, 501), 9, BF))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, run()))


def test_python_refusals(cuda_lib):
    rlk = cuda_lib
    x, w, b = randn((8, 16), 1, BF), randn((4, 16), 2, BF), randn((4,), 3)
    z = randn((8, 4), 4, BF)
    for bad in (lambda: rlk.gated_linear(x.float(), w, w), lambda: rlk.gated_linear(x, w, w[:3]), lambda: rlk.gated_linear(x, w[:, :8], w[:, :8]),
                lambda: rlk.gated_linear(x.cpu(), w, w), lambda: rlk.gated_linear(x, w, w, b, b.to(BF)), lambda: rlk.gated_linear(x, w, w, b[:3]),
                lambda: rlk.gated_linear(x, w, w, out=torch.empty(8, 5, device="cuda")), lambda: rlk.gated_linear(x, w.t().contiguous().t(), w),
                lambda: rlk.gated_linear(x, w, w, out_dtype=torch.float16),
                lambda: rlk.gated_linear_backward(z, x, w, w, z[:7], z), lambda: rlk.gated_linear_backward(z, x[:7], w, w, z, z),
                lambda: rlk.gated_linear_backward(z, x, w, w, z, z, accumulate=True),
                lambda: rlk.gated_linear_backward(z, x, w, w, z, z, grad_w_gate=torch.empty(4, 16, device="cuda"), grad_w_up=torch.empty(4, 16, device="cuda", dtype=BF))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(rlk.RlkError):
        rlk.gated_linear(x, w, w, activation=9)
    with pytest.raises(rlk.RlkError):
        rlk.gated_linear_backward(z, None, w, w, z, z)                # the weights' gradients need x
    odd = randn((8, 17), 5, BF)[:, 1:]
    with pytest.raises(rlk.RlkError):                                  # a workspace too short for the copy
        rlk.gated_linear(odd, w, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# one tile a CTA, its K whole and split; pairs with one and with several tiles
@pytest.mark.parametrize("M,N,K", [(40, 64, 130), (100, 300, 512), (3000, 1500, 250), (6000, 3100, 128)])
@pytest.mark.parametrize("stage", [0, 1])
def test_waits_that_run_out(cuda_lib, M, N, K, stage):
    """The call returns once its copies are there, what depended on them is NaN, the next call is clean."""
    rlk = cuda_lib
    x, wg, wu = randn((M, K), 1, BF), randn((N, K), 2, BF, 0.05), randn((N, K), 3, BF, 0.05)
    want = rlk.gated_linear(x, wg, wu, out_dtype=F32)
    torch.cuda.synchronize()
    rlk.set_wait_limit(2_000_000)   # about a millisecond
    try:
        rlk.withhold_copy(stage)
        got = rlk.gated_linear(x, wg, wu, out_dtype=F32)
        torch.cuda.synchronize()
    finally:
        rlk.withhold_copy(-1)
        rlk.set_wait_limit(0)
    nan = torch.isnan(got)
    assert bool(nan[0, 0]) and torch.equal(got[~nan], want[~nan])
    for _ in range(3):
        assert torch.equal(rlk.gated_linear(x, wg, wu, out_dtype=F32), want)
