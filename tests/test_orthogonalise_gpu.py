"""Orthogonalised updates against the iteration in 64 bits.

Tolerances.  The result's rounding to bf16 is 2^-8 of an entry at most, so of the norm.
Up to 128 on the shorter side the operands have 22 bits: to first order a singular
value s is moved in a step by (|b A + 2 c A^2| + 2 |P|) / |a + P| u of it (A, P and X
rounded to u; A = s^2, P = b A + c A^2), and what is off before a step is multiplied by
|a + 3 b A + 5 c A^2| / |a + P|.  Summed over 5 steps, the worst s in [0.001, 1] gives 109 u, over 8
460 u: with u = 2^-21 0.0003 at most, and sums in fp32 (2^-23 of sum |a b|, |a b| up to
sqrt(n) times the sum) about as much.  So 2^-8 + 0.001.
Above 128, u = 2^-11 gives 0.053 for the worst direction if all roundings push it the
same way.  A matrix of more than 128 directions with independent errors of either sign is
off by their root mean square: roundings are u / sqrt(3) at most in that sense and those of
15 products add as squares, median 15 u (not 109): 15 / sqrt(15) / sqrt(3) u = 0.0011, beside the
bf16 rounding's 0.0017 (at most 2^-8).  So 2^-8 + 0.0011, and 0.06 for the largest entry.
"""
import pytest
import torch

from _layers import randn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ABC = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def orth64(g, steps=5, abc=ABC, eps=EPS):
    a, b, c = abc
    x = g.double()
    x = x / (x.norm(dim=(-2, -1), keepdim=True) + eps)
    turned = x.shape[-2] > x.shape[-1]
    x = x.transpose(-2, -1) if turned else x
    for _ in range(steps):
        p = x @ x.transpose(-2, -1)
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.transpose(-2, -1) if turned else x


def check(got, want):
    rel, largest = 2 ** -8 + (0.001 if min(want.shape[-2:]) <= 128 else 0.0011), 0.06
    d = got.double() - want
    norm = want.norm(dim=(-2, -1))
    assert torch.isfinite(got).all()
    assert bool((d.norm(dim=(-2, -1)) <= rel * norm).all()), (d.norm(dim=(-2, -1)) / norm).max()
    rms = want.square().mean().sqrt()
    assert ((d.abs() / want.abs().clamp_min(rms)).max() <= largest), (d.abs() / want.abs().clamp_min(rms)).max()


def low_rank(shape, seed, dtype):
    B, m, n = shape
    r = max(1, min(m, n) // 16)
    x = randn((B, m, r), seed) @ randn((B, r, n), seed + 1) / r ** 0.5 + 0.05 * randn(shape, seed + 2)
    return (1e-3 * x).to(dtype)


SHAPES = [(1, 1, 1), (1, 1, 9), (1, 7, 1), (2, 3, 5), (1, 64, 64), (3, 65, 63), (1, 128, 300), (2, 300, 129), (1, 257, 1000), (1, 1000, 257), (1, 512, 512), (24, 130, 200),
          (1, 2000, 1700), (1, 1700, 2300), (5, 640, 520), (3, 256, 256), (2, 255, 700), (2, 129, 129),
          (1, 1003, 2731), (1, 2731, 1003), (1, 900, 1000), (1, 2600, 2700), (30, 300, 400), (30, 400, 300)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("make", [lambda s, k, t: randn(s, k, t), low_rank], ids=["noise", "low_rank"])
def test_shapes(cuda_lib, shape, dtype, make):
    g = make(shape, 3, dtype)
    got = cuda_lib.orthogonalise(g)
    assert got.dtype == BF and got.shape == g.shape
    check(got, orth64(g))
    if shape[0] == 1:
        assert torch.equal(cuda_lib.orthogonalise(g[0]), got[0])


@pytest.mark.parametrize("steps,abc", [(1, ABC), (2, ABC), (3, (1.875, -1.25, 0.375)), (8, ABC), (6, (1.5, -0.5, 0.0)), (1, (0.0, 0.0, 1.0)), (1, (1.0, 0.0, 0.0)), (1, (0.0, 1.0, 0.0))])
def test_steps_and_coefficients(cuda_lib, steps, abc):
    for m, n in ((96, 200), (200, 96)):
        q = torch.linalg.qr(randn((200, 96), 1).double())[0]
        g = (q * torch.linspace(0.2, 1.0, 96, dtype=torch.float64, device="cuda")).float()   # singular values between 0.2 and 1
        g = (g if m > n else g.t()).contiguous()
        check(cuda_lib.orthogonalise(g, steps=steps, coefficients=abc), orth64(g, steps, abc))


def test_singular_values_go_to_one(cuda_lib):
    g = randn((300, 700), 5)
    for steps in (5, 12):
        s = torch.linalg.svdvals(cuda_lib.orthogonalise(g, steps=steps).double())
        assert s.min() > 0.6 and s.max() < 1.3    # the polynomial's range once a value has come near 1: 0.68 to 1.2


def test_strides_and_in_place(cuda_lib):
    rlk = cuda_lib
    for dtype in (BF, F32):
        for lead in (0, 1, 3):
            wide = torch.full((4, 50, 90), float("nan"), dtype=dtype, device="cuda")
            g = wide[:, 5:45, lead:lead + 77]
            g.copy_(randn((4, 40, 77), 2))
            want = rlk.orthogonalise(g.contiguous())
            room = torch.full((4, 60, 101), 7.0, dtype=BF, device="cuda")
            out = room[:, 3:43, lead:lead + 77]
            assert rlk.orthogonalise(g, out=out) is out and torch.equal(out, want)
            seen = torch.zeros_like(room, dtype=torch.bool)
            seen[:, 3:43, lead:lead + 77] = True
            assert (room[~seen] == 7).all()                            # nothing beside it
            rows = rlk.orthogonalise(g[:, ::2])                        # every second row
            assert torch.equal(rows, rlk.orthogonalise(g[:, ::2].contiguous()))
            if dtype == BF:
                assert rlk.orthogonalise(g, out=g) is g and torch.equal(g, want)
    same = randn((1, 30, 20), 4).expand(3, 30, 20)                     # one matrix three times
    got = rlk.orthogonalise(same)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    # from one matrix of a row or a column
    row, col = randn((1, 33), 5), randn((33, 1), 6)
    assert torch.allclose(rlk.orthogonalise(row).double(), orth64(row), rtol=0.02) and torch.allclose(rlk.orthogonalise(col).double(), orth64(col), rtol=0.02)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-7, 1.0, 1e18, 1e25, 1e37])
def test_sizes_of_numbers(cuda_lib, size):
    """The result does not depend on the size of the numbers (with eps 0)."""
    for dtype in (BF, F32):
        g = (randn((40, 64), 1).clamp(-3, 3).double() * size).to(dtype)
        check(cuda_lib.orthogonalise(g, eps=0.0), orth64(g, eps=0.0))
    mixed = randn((40, 64), 1) * torch.logspace(-30, 30, 64, device="cuda")
    check(cuda_lib.orthogonalise(mixed), orth64(mixed))


def test_eps(cuda_lib):
    g = randn((40, 64), 1) * 1e-9
    check(cuda_lib.orthogonalise(g, eps=1e-7), orth64(g, eps=1e-7))
    z = torch.zeros(3, 20, 30, device="cuda")
    z[1] = randn((20, 30), 1)
    for eps in (0.0, 1e-7):
        got = cuda_lib.orthogonalise(z, eps=eps)
        assert (got[[0, 2]] == 0).all() and torch.isfinite(got).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape", [(4, 70, 90), (3, 300, 200), (40, 260, 270)])
def test_a_bad_matrix_leaves_the_others(cuda_lib, bad, shape):
    g = randn(shape, 1)
    want = cuda_lib.orthogonalise(g)
    g[1, 5, 7] = bad
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = cuda_lib.orthogonalise(g, status_word=word)
    assert word.item() == cuda_lib.STATUS_NONFINITE and torch.isnan(got[1]).all()
    rest = torch.arange(shape[0]) != 1
    assert torch.equal(got[rest], want[rest])
    cuda_lib.orthogonalise(want, status_word=word.zero_())
    assert word.item() == 0


def test_streams_graph_and_repeat(cuda_lib):
    rlk = cuda_lib
    g = randn((3, 300, 520), 1)
    want = rlk.orthogonalise(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = rlk.orthogonalise(g)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = rlk.orthogonalise(g)
    g.copy_(randn((3, 300, 520), 2))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, rlk.orthogonalise(g))


def test_refusals(cuda_lib):
    rlk = cuda_lib
    g = randn((8, 16), 1)
    for bad in (lambda: rlk.orthogonalise(g.cpu()), lambda: rlk.orthogonalise(g.half()), lambda: rlk.orthogonalise(g[0]), lambda: rlk.orthogonalise(g.t()),
                lambda: rlk.orthogonalise(g, out=torch.empty(8, 16, device="cuda")), lambda: rlk.orthogonalise(g, out=torch.empty(8, 15, dtype=BF, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (dict(steps=0), dict(steps=65), dict(coefficients=(17.0, 0.0, 0.0)), dict(coefficients=(float("nan"), 0.0, 0.0)), dict(eps=-1.0), dict(eps=float("inf")),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(rlk.RlkError):
            rlk.orthogonalise(g, **bad)
    assert rlk.orthogonalise(torch.empty(0, 8, 16, device="cuda")).shape == (0, 8, 16)


@pytest.mark.parametrize("shape", [(1, 100, 130), (1, 900, 700), (6, 1024, 1024)])
def test_waits_that_run_out(cuda_lib, shape):
    """The call returns, what depended on the wait is NaN, and the next call is clean."""
    rlk = cuda_lib
    g = randn(shape, 1)
    want = rlk.orthogonalise(g)
    torch.cuda.synchronize()
    rlk.set_wait_limit(2_000_000)   # about a millisecond
    try:
        rlk.withhold_copy(0)
        got = rlk.orthogonalise(g)
        torch.cuda.synchronize()
    finally:
        rlk.withhold_copy(-1)
        rlk.set_wait_limit(0)
    assert torch.isnan(got).any()
    for _ in range(3):
        assert torch.equal(rlk.orthogonalise(g), want)


# up to 128 x 1024 and its transpose, one kernel: one to eight CTAs, 128 of the longer side each
SMALL = [(1, 128, 128), (1, 128, 1024), (1, 1024, 128), (2, 5, 1000), (2, 1000, 5), (40, 100, 260), (40, 260, 100), (1, 90, 897), (1, 897, 90),
         (3, 640, 17), (3, 17, 640), (1, 385, 128), (1, 128, 511), (200, 65, 70), (1, 1, 1024), (1, 1024, 1), (1, 128, 1025), (1, 1025, 128), (1, 129, 130),
         (2, 100, 800), (2, 800, 100), (2, 33, 700), (2, 700, 33)]


@pytest.mark.parametrize("shape", SMALL, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("make", [lambda s, k, t: randn(s, k, t), low_rank], ids=["noise", "low_rank"])
def test_small_shapes(cuda_lib, shape, dtype, make):
    g = make(shape, 4, dtype)
    got = cuda_lib.orthogonalise(g)
    check(got, orth64(g))
    assert torch.equal(cuda_lib.orthogonalise(g), got)
    assert torch.equal(cuda_lib.orthogonalise(g[-1]), got[-1])


@pytest.mark.parametrize("shape", [(3, 128, 1000), (3, 1000, 128), (150, 30, 500), (150, 500, 30)])
@pytest.mark.parametrize("steps", [1, 2, 8])
def test_small_in_place_strided_and_captured(cuda_lib, shape, steps):
    rlk = cuda_lib
    B, m, n = shape
    for lead in (0, 3):
        room = torch.full((B, m + 2, n + 11), 7.0, dtype=BF, device="cuda")
        g = room[:, 1:m + 1, lead:lead + n]
        g.copy_(randn(shape, 5))
        want = rlk.orthogonalise(g.contiguous(), steps=steps)
        check(want, orth64(g, steps))
        kept = g.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rlk.orthogonalise(g, steps=steps, out=g)
        for _ in range(2):
            g.copy_(kept)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(g, want)
        seen = torch.zeros_like(room, dtype=torch.bool)
        seen[:, 1:m + 1, lead:lead + n] = True
        assert (room[~seen] == 7).all()


@pytest.mark.parametrize("shape", [(4, 100, 1000), (4, 1000, 100), (170, 128, 128)])
def test_a_bad_small_matrix_leaves_the_others(cuda_lib, shape):
    g = randn(shape, 1)
    want = cuda_lib.orthogonalise(g)
    g[1, -1, -1] = float("nan")
    got = cuda_lib.orthogonalise(g)
    rest = torch.arange(shape[0]) != 1
    assert torch.isnan(got[1]).all() and torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("shape", [(1, 100, 100), (3, 120, 1024), (3, 1024, 120), (170, 60, 250)])
def test_small_waits_that_run_out(cuda_lib, shape):
    """The first matrix is NaN, whichever of its CTAs gave up; the others and the next call are right."""
    rlk = cuda_lib
    g = randn(shape, 1)
    want = rlk.orthogonalise(g)
    torch.cuda.synchronize()
    rlk.set_wait_limit(2_000_000)   # about a millisecond
    try:
        rlk.withhold_copy(0)
        got = rlk.orthogonalise(g)
        torch.cuda.synchronize()
    finally:
        rlk.withhold_copy(-1)
        rlk.set_wait_limit(0)
    assert torch.isnan(got[0]).all() and torch.equal(got[1:], want[1:])
    for _ in range(3):
        assert torch.equal(rlk.orthogonalise(g), want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("exponent", [-41, 39, 126, -120])
def test_many_numbers_of_one_size(cuda_lib, dtype, exponent):
    """2^26 numbers on one side of a range's border: their sums of squares stay in fp32, and a power of two changes nothing."""
    g = torch.where(randn((65536, 1024), 1, dtype) > 0, 1.875, -1.875).to(dtype)
    assert torch.equal(cuda_lib.orthogonalise(g * 2.0 ** exponent, eps=0.0), cuda_lib.orthogonalise(g, eps=0.0))


def test_least_numbers(cuda_lib):
    """Below 2^-126: a power of two's multiples of the least fp32 number are exact, and so are their squares' sums."""
    q = torch.randint(-8, 9, (64, 96), generator=torch.Generator().manual_seed(1)).float().cuda()
    q[0, 0] = 8.0
    check(cuda_lib.orthogonalise(q * 2.0 ** -149, eps=0.0), orth64(q, eps=0.0))
