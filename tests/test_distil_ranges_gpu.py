"""The ends of the ranges of a distillation step's operators: more rows than a grid's side, every named place in use,
ties in each form that a row is read in, element offsets past 32 bits."""
import pytest
import torch

from _distil import act64, tokens_grad64
from _layers import EPS32, HALF_ULP, randn
from test_orthogonalise_gpu import check as check_orth, orth64
from test_token_logprobs_gpu import check, given, logits, odd_layout

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_more_rows_than_a_grid_has(cuda_lib, dtype):
    rlk, T, V, C, top = cuda_lib, 140001, 37, 2, 3
    z, ids = logits(T, V, dtype, 1), given(T, V, C, 1)
    state = rlk.new_token_state(T, "cuda")
    lp, h, ti, tl = rlk.token_logprobs(z, ids, 0.9, n_top=top, state=state)
    glp, gh, gt = randn((T, C), 2), randn((T,), 3), randn((T, top), 4)
    dz = rlk.token_logprobs_backward(z, ids, 0.9, state, glp, gh, top_ids=ti, grad_top=gt)
    keep = torch.tensor([0, 1, 65534, 65535, 65536, 131069, 131070, T - 1])
    check(rlk, z[keep], ids[keep], 0.9, top)
    for a, b in zip((lp, h, ti, tl), rlk.token_logprobs(z[keep], ids[keep], 0.9, n_top=top)):
        assert torch.equal(a[keep], b)
    want, terms = tokens_grad64(z[keep], ids[keep], 0.9, glp[keep], gh[keep], ti[keep], gt[keep])
    tol = terms * 340 * EPS32 + want.abs() * HALF_ULP[dtype] * 1.01
    assert ((dz[keep].double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["levels", "flat", "up", "down", "few", "lowest"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,odd", [(3, 70001, False), (100, 70001, True), (320, 17003, True)], ids=["four_ctas", "two_ctas", "ring"])
def test_ties_in_every_form(cuda_lib, kind, dtype, T, V, odd):
    """The largest number of alternatives, long ties and sorted rows, in rows that CTAs share and in the ring."""
    z = logits(T, V, dtype, V, kind)
    z = odd_layout(z) if odd else z
    ids = given(T, V, 2, 5)
    keep = torch.tensor([0, T // 2, T - 1])
    all_ = cuda_lib.token_logprobs(z, ids, 1.3, n_top=128)
    part = cuda_lib.token_logprobs(z[keep], ids[keep], 1.3, n_top=128)
    for a, b in zip(all_, part):
        assert torch.equal(a[keep].view(torch.int32), b.view(torch.int32))
    check(cuda_lib, z[keep], ids[keep], 1.3, 128)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 9001])
def test_every_named_place(cuda_lib, dtype, V):
    """1024 tokens and 128 alternatives a row, most of them named several times."""
    rlk, T, C, top = cuda_lib, 3, 1024, 128
    z, ids = logits(T, V, dtype, 2), given(T, min(V, 200), C, 2)
    state = rlk.new_token_state(T, "cuda")
    ti = rlk.token_logprobs(z, ids, 0.8, n_top=top, state=state)[2]
    ids[:, :top] = ti                                                  # what the alternatives name too
    glp, gh, gt = randn((T, C), 2), randn((T,), 3), randn((T, top), 4)
    dz = rlk.token_logprobs_backward(z, ids, 0.8, state, glp, gh, top_ids=ti, grad_top=gt, grad_dtype=F32)
    want, terms = tokens_grad64(z, ids, 0.8, glp, gh, ti, gt)
    rel = (V / 1024 + 40 + 4 * 60 + 24 + 2 * (C + top)) * EPS32
    assert ((dz.double().cpu() - want).abs() <= terms * rel + want.abs() * EPS32 * 1.01 + 1e-37).all()


def test_gated_offsets_past_32_bits(cuda_lib):
    """y, the projections, dy and dx of more than 2^32 bytes: the last rows as they are alone."""
    rlk, M, N, K, R = cuda_lib, 320000, 7168, 64, 300
    x, wg, wu = randn((M, K), 1, BF16), randn((N, K), 2, BF16, 0.1), randn((N, K), 3, BF16, 0.1)
    y, g, u = rlk.gated_linear(x, wg, wu, return_preact=True)
    for rows in (slice(0, R), slice(M - R, M)):
        zg, zu = x[rows].double() @ wg.double().t(), x[rows].double() @ wu.double().t()
        for got, want in ((g, zg), (u, zu), (y, act64(zg, rlk.ACT_SILU)[0] * zu)):
            # sums of 64 products are off by 2 K e of their sizes (below 30 here), act by as much, then half an ulp
            assert ((got[rows].double() - want).abs() <= HALF_ULP[BF16] * want.abs() + 1e-3).all()
    dy = y                                                             # any rows will do
    want_x, want_g, want_u = (torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((0, K), (N, K), (N, K)))
    dx, dwg, dwu, dbg, dbu = rlk.gated_linear_backward(dy, x, wg, wu, g, u)
    for r in range(0, M, 20000):
        v, s = act64(g[r:r + 20000], rlk.ACT_SILU)
        d = dy[r:r + 20000].double()
        dg, du = d * u[r:r + 20000].double() * s, d * v
        want_g += dg.t() @ x[r:r + 20000].double()
        want_u += du.t() @ x[r:r + 20000].double()
        if r + 20000 >= M:
            want_x = dg @ wg.double() + du @ wu.double()
            size = dg.abs() @ wg.double().abs() + du.abs() @ wu.double().abs()
            assert ((dx[r:].double() - want_x).abs() <= HALF_ULP[BF16] * (want_x.abs() + 1.1 * size)).all()
    for got, want in ((dwg, want_g), (dwu, want_u)):
        # roundings of dg and du of either sign, M of them: far below half an ulp of the norm
        assert (got.double() - want).norm() <= 2 ** -8 * want.norm()
    assert torch.isfinite(dbg).all() and torch.isfinite(dbu).all()


@pytest.mark.parametrize("shape,dtype", [((65535, 128, 256), F32), ((40000, 120, 500), BF16), ((5000, 1000, 500), BF16)], ids=["one_kernel", "small_launches", "launches"])
def test_orthogonalise_offsets_past_32_bits(cuda_lib, shape, dtype):
    g = torch.randn(shape, dtype=dtype, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    got = cuda_lib.orthogonalise(g)
    for b in (0, shape[0] // 2, shape[0] - 1):
        check_orth(got[b:b + 1], orth64(g[b:b + 1]))


def test_the_most_matrices(cuda_lib):
    rlk = cuda_lib
    g = randn((65535, 6, 10), 1)
    got = rlk.orthogonalise(g)
    check_orth(got[::5000], orth64(g[::5000]))
    assert torch.equal(got[-1], rlk.orthogonalise(g[-1]))


@pytest.mark.parametrize("shape", [(1, 65536, 3), (1, 3, 65536), (2, 65536, 130), (2, 130, 65536)], ids=str)
def test_the_longest_sides(cuda_lib, shape):
    g = randn(shape, 1)
    check_orth(cuda_lib.orthogonalise(g), orth64(g))
