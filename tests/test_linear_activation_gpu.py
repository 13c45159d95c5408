"""The linear layer's activations far from zero: fp32 outputs and slopes by their
relative error, whatever the path (dot products, one tile, pairs' tiles).

A pre-activation is one bf16 product here, so it is exact.  With e = 2^-24, GELU's
exponential has an exponent of z^2 / 2 from three roundings (1.5 z^2 e), SiLU's one of |z|
from two (1.5 |z| e).  The hardware's exponential and reciprocal are good to 4 e and 2 e;
what is left (a polynomial of degree 7 or a sum, four products) stays below 16 e.  So
(2 z^2 + 24) e and (2 |z| + 24) e.  GELU's slope left of -4 is a difference of
terms that are 17/15 of it together.
"""
import pytest
import torch

from _layers import EPS32 as E, HALF_ULP, act64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def all_bf16(lo, hi):
    """Every bf16 number of [lo, hi], both positive, and its negative."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    v = (bits << 16).view(F32)
    v = v[(v >= lo) & (v <= hi)]
    return torch.cat([-v.flip(0), v]).to(BF).cuda()


def near(got, want, rel, what):
    d = (got.double() - want).abs() / want.abs()
    assert bool((d <= rel).all()), f"{what}: {(d / rel).max().item():.3g} of the bound"


ACTS = {"gelu": (1, lambda z: (2 * z * z + 24) * E, 12.0), "silu": (2, lambda z: (2 * z.abs() + 24) * E, 80.0)}


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 3, 8, 2000])
@pytest.mark.parametrize("out", [F32, BF])
def test_values(cuda_lib, act, M, out):
    code, rel, top = ACTS[act]
    z = all_bf16(2.0 ** -6, top)
    if M > 1000:
        z = z.repeat(4)
    y = cuda_lib.linear(torch.ones(M, 1, dtype=BF, device="cuda"), z[:, None], activation=code, out_dtype=out)
    zd = z.double()
    near(y, act64(z, code)[0].expand(M, -1), (1 + HALF_ULP[out]) * rel(zd) + HALF_ULP[out], act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("odd", [False, True])
def test_slopes(cuda_lib, act, odd):
    """A single row's bias gradient is dy act'(z), unrounded."""
    code, rel, top = ACTS[act]
    z = all_bf16(4.0, top)
    z = z[: len(z) // 8 * 8 - odd][None]
    dy, x = torch.ones_like(z), torch.ones(1, 8, dtype=BF, device="cuda")
    db = cuda_lib.linear_backward(dy, x, torch.ones(z.shape[1], 8, dtype=BF, device="cuda"), z, activation=code)[2]
    zd = z[0].double()
    near(db, act64(z[0], code)[1], 17 / 15 * rel(zd) + E, act)
