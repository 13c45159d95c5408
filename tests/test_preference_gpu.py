"""The paired preference loss against its plain 64-bit form.

Tolerances: the sums are double-floats, so a reward carries the rounding of the
token differences (half an ulp each) and of three fp32 operations:
|r| error <= beta sum_t e (|logp| + |ref|) + 4 e |r|; the loss and the slope are
1-Lipschitz in h (sigmoid, hinge) or 2 |d| / beta (IPO), plus the
few-ulp error of expf / log1pf (8 e relative, 2 e absolute).
"""
import math

import numpy as np
import pytest
import torch

from _layers import EPS32 as E, preference64, randn

pytestmark = pytest.mark.gpu

KINDS = {"sigmoid": 0, "ipo": 1, "hinge": 2}


def batch(lens, seed, masked=0.15, empty=()):
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n = int(off[-1])
    lp = -randn((n,), seed).abs() * 1.5
    ref = lp + randn((n,), seed + 1, scale=0.1)
    rng = np.random.default_rng(seed)
    m = (rng.random(n) >= masked).astype(np.uint8)
    for s in empty:
        m[off[s]:off[s + 1]] = 0
    return lp, ref, torch.from_numpy(m).cuda(), torch.from_numpy(off).cuda(), off


def check(rlk, lp, ref, mask, off, offh, kind, beta, smoothing, margin, mean):
    loss, grad, reward, stats = rlk.preference_loss(lp, ref, off, loss_mask=mask, loss_type=KINDS[kind], beta=beta,
                                                    label_smoothing=smoothing, margin=margin, length_normalise=mean)
    L, G, R, S = preference64(lp, ref, mask, offh, KINDS[kind], beta, smoothing, margin, mean)
    P = max(1, (len(offh) - 1) // 2)
    mag = lp.double().abs().cpu() + (0 if ref is None else ref.double().abs().cpu())
    if mask is not None:
        mag = torch.where(mask.cpu() != 0, mag, 0.0)
    dr = torch.zeros_like(R)
    for s in range(len(R)):
        n = max(1, int(offh[s + 1] - offh[s])) if mean else 1
        dr[s] = beta * E * mag[offh[s]:offh[s + 1]].sum() / (n if mean and mask is None else 1) + 4 * E * R[s].abs() + 1e-12
    assert bool(((reward.cpu().double() - R).abs() <= dr).all())
    dh = (dr[0::2] + dr[1::2]) + 3 * E * (R[0::2].abs() + R[1::2].abs() + abs(margin))
    h = R[0::2] - R[1::2] - margin
    if kind == "ipo":
        d = (h - 0.5) / beta
        dl, ds = 2 * d.abs() * dh / beta + (dh / beta) ** 2 + 8 * E * d * d, 2 * dh / beta ** 2 + 8 * E * d.abs() / beta
    else:
        dl, ds = dh + 8 * E * (h.abs() + 1) + 2 * E, dh + 10 * E
    assert abs(loss.item() - L) <= dl.sum().item() / P + 4 * E * abs(L) + 1e-12
    per = torch.zeros_like(G)
    for s in range(len(R)):
        i = slice(int(offh[s]), int(offh[s + 1]))
        per[i] = beta * ds[s // 2] / P * (1 if not mean else 1 / max(1, int((mask.cpu()[i] != 0).sum()) if mask is not None else i.stop - i.start))
    assert bool(((grad.cpu().double() - G).abs() <= per + 6 * E * G.abs() + 1e-14).all())
    if mask is not None:
        assert bool((grad.cpu()[mask.cpu() == 0] == 0).all())
    st = stats.cpu().double()
    assert st[1] == S[1] and abs(st[2] - S[2]) < 1e-6
    assert bool(((st[3:] - S[3:]).abs() <= dr.max() * 2 + 8 * E * (R.abs().max() if len(R) else 0) + 1e-12).all())


LENS = {
    "one_token_each": [1, 1], "short": [3, 5, 1, 9], "with_zero_lengths": [0, 7, 4, 0, 0, 0, 12, 3],
    "segment_edges": [2047, 2048, 2049, 4096, 4097, 1, 6143, 6145], "long": [30011, 17, 9000, 20000],
    "many": [int(v) for v in np.random.default_rng(5).integers(1, 300, 600)],
}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("kind,beta,smoothing,margin", [("sigmoid", 0.1, 0.0, 0.0), ("sigmoid", 0.5, 0.2, 0.3), ("ipo", 0.1, 0.0, 0.0),
                                                        ("hinge", 0.1, 0.0, -0.2)])
@pytest.mark.parametrize("mean,ref", [(False, True), (True, False)])
def test_matches_the_plain_form(cuda_lib, lens, kind, beta, smoothing, margin, mean, ref):
    lp, rf, m, off, offh = batch(LENS[lens], 3, empty=(1,) if len(LENS[lens]) > 4 else ())
    for mask in (m, None):
        check(cuda_lib, lp, rf if ref else None, mask, off, offh, kind, beta, smoothing, margin, mean)


def test_gradient_against_differences(cuda_lib):
    lp, rf, m, off, offh = batch([9, 14, 30, 2, 5, 5], 11)
    for kind in KINDS:
        _, g, _, _ = cuda_lib.preference_loss(lp, rf, off, loss_mask=m, loss_type=KINDS[kind], beta=0.3)
        v = randn((lp.numel(),), 12).double().cpu()
        f = lambda s: preference64(lp.double().cpu() + s * v, rf, m, offh, KINDS[kind], 0.3, 0.0, 0.0, False)[0]
        want, got = (f(1e-5) - f(-1e-5)) / 2e-5, (g.cpu().double() * v).sum().item()
        assert abs(got - want) <= 1e-5 * (g.cpu().double() * v).abs().sum().item() + 1e-7


def test_masked_tokens_are_never_looked_at(cuda_lib):
    lp, rf, m, off, _ = batch([40, 33, 21, 50], 13, masked=0.4)
    want = cuda_lib.preference_loss(lp, rf, off, loss_mask=m)
    lp2, rf2 = lp.clone(), rf.clone()
    lp2[m == 0], rf2[m == 0] = -math.inf, math.nan
    got = cuda_lib.preference_loss(lp2, rf2, off, loss_mask=m)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_infinities_go_through_the_formula(cuda_lib):
    lp, rf, _, off, _ = batch([10, 12, 9, 9, 3000, 2500], 14)
    for at, loss_inf in ((4, True), (15, False)):       # in a chosen response; in a rejected one
        x = lp.clone()
        x[at] = -math.inf
        loss, grad, reward, stats = cuda_lib.preference_loss(x, rf, off)
        assert math.isinf(loss.item()) == loss_inf and not math.isnan(loss.item())
        assert reward[0 if loss_inf else 1].item() == -math.inf
        assert torch.isfinite(grad).all()
        assert grad[0].item() == pytest.approx(float(-np.float32(0.1) / np.float32(3)) if loss_inf else 0.0, abs=1e-9)   # beta is an fp32
    x = lp.clone()
    x[4] = math.nan
    loss, grad, reward, _ = cuda_lib.preference_loss(x, rf, off)
    assert math.isnan(loss.item()) and torch.isnan(grad[:22]).all() and torch.isfinite(grad[22:]).all()
    for kind in (0, 1, 2):                               # large rewards overflow nothing
        x = lp.clone()
        x[0], x[10] = 1e4, -1e4
        out = cuda_lib.preference_loss(x, rf, off, loss_type=kind)
        assert all(torch.isfinite(t).all() for t in out)


@pytest.mark.parametrize("offsets", [[0, 10, 5, 20, 40], [0, 10, 20, 30, 41], [-1, 10, 20, 30, 40], [0, 10, 20, 2 ** 31 - 1, 40],
                                     [30, 20, 10, 5, 0]])
def test_invalid_offsets_give_nan_and_stay_inside(cuda_lib, offsets):
    n, pad = 40, 256
    buf = torch.full((n + 2 * pad,), -1.0, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    loss, grad, reward, stats = cuda_lib.preference_loss(buf[pad:pad + n], None, off)
    assert all(torch.isnan(t).all() for t in (loss, grad, reward, stats))


def test_no_pairs_and_tokens_outside(cuda_lib):
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, grad, reward, stats = cuda_lib.preference_loss(torch.ones(7, device="cuda"), None, off)
    assert loss.item() == 0 and bool((grad == 0).all()) and reward.numel() == 0 and stats[1].item() == 0
    lp = -randn((30,), 2).abs()
    off = torch.tensor([4, 10, 22], dtype=torch.int32, device="cuda")
    _, g, _, _ = cuda_lib.preference_loss(lp, None, off)
    inner = cuda_lib.preference_loss(lp[4:22].clone(), None, off - 4)[1]
    assert torch.equal(g[4:22], inner) and bool((g[:4] == 0).all()) and bool((g[22:] == 0).all())


def test_a_sequence_does_not_depend_on_the_batch(cuda_lib):
    lens = [5000, 3000, 100, 2500, 9000, 8000]
    lp, rf, m, off, offh = batch(lens, 17)
    _, _, reward, _ = cuda_lib.preference_loss(lp, rf, off, loss_mask=m)
    for p in range(3):
        a, b = int(offh[2 * p]), int(offh[2 * p + 2])
        sub = (off[2 * p:2 * p + 3] - a).contiguous()
        r = cuda_lib.preference_loss(lp[a:b].clone(), rf[a:b].clone(), sub, loss_mask=m[a:b].clone())[2]
        assert torch.equal(r, reward[2 * p:2 * p + 2])


def test_repeats_and_captures(cuda_lib):
    lp, rf, m, off, _ = batch([int(v) for v in np.random.default_rng(7).integers(10, 2500, 64)], 19)
    want = cuda_lib.preference_loss(lp, rf, off, loss_mask=m)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = cuda_lib.preference_loss(lp, rf, off, loss_mask=m)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
