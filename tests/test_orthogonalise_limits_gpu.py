"""How far an iteration may grow: fp16 holds the entries of A and P = b A + c A A up to 63.97 (65504 / 2^10).
Inside that the result is the iteration's, past it the result is not finite and the status word says so."""
import pytest
import torch

from _layers import randn
from test_orthogonalise_gpu import check, orth64

pytestmark = pytest.mark.gpu
# one kernel with one and with several CTAs a matrix; products of their own: all of A, its blocks of 128, of 256
SHAPES = [(64, 64), (40, 200), (200, 40), (300, 300), (500, 500), (700, 300), (300, 700), (950, 1300), (900, 5000), (5000, 900)]


def run(rlk, g, steps, abc):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    return rlk.orthogonalise(g, steps=steps, coefficients=abc, status_word=word), word.item()


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("norm,inside", [(7.9, True), (8.1, False)])
def test_norms_of_rows(cuda_lib, m, n, norm, inside):
    """Equal singular values, multiplied by a in each step (P = 0): before the third they are `norm`,
    A's diagonal norm^2 = 62.4 or 65.6, and X's own entries far below 64."""
    r = min(m, n)
    q = torch.linalg.qr(randn((max(m, n), r), 1).double())[0].float()
    g = (q if m > n else q.t()).contiguous()
    a = (norm * r ** 0.5) ** 0.5                       # 1 / sqrt(r) a a = norm
    assert a <= 16 and a * a / r ** 0.5 * g.abs().max() < 8
    got, word = run(cuda_lib, g, 3, (a, 0.0, 0.0))
    if inside:
        assert word == 0
        check(got, orth64(g, 3, (a, 0.0, 0.0)))
    else:
        assert word == cuda_lib.STATUS_NONFINITE and not torch.isfinite(got).all()


@pytest.mark.parametrize("m,n", SHAPES + [(2100, 2200), (2200, 2100)])
@pytest.mark.parametrize("a,inside", [(0.5, True), (0.9, False)])
def test_entries_of_p(cuda_lib, m, n, a, inside):
    """One singular value: 1, then s = a + 2.  A = s^2 is 6.3 or 8.4, P = s^2 + s^4 45.3 or 79.1."""
    g = torch.zeros(m, n, device="cuda")
    g[m // 2, n // 3] = 3.0
    got, word = run(cuda_lib, g, 2, (a, 1.0, 1.0))
    if inside:
        assert word == 0
        want = orth64(g, 2, (a, 1.0, 1.0))
        assert ((got.double() - want).abs() <= (2 ** -8 + 0.001) * want.abs()).all()
    else:
        assert word == cuda_lib.STATUS_NONFINITE and not torch.isfinite(got).all()


@pytest.mark.parametrize("shape", [(3, 60, 70), (3, 300, 200), (3, 259, 301), (3, 1030, 1500)])
def test_a_matrix_that_grows_too_far_leaves_the_others(cuda_lib, shape):
    """Only the second matrix passes the limit: the others keep their bits; rows on and off 16 bytes."""
    rlk, abc = cuda_lib, (0.9, 1.0, 1.0)
    B, m, n = shape
    g = 1e-3 * randn(shape, 3)                          # many singular values below 1: their P stays small
    want, word = run(rlk, g, 2, abc)
    assert word == 0 and torch.isfinite(want).all()
    g[1] = 0.0
    g[1, 5, 7] = 1.0
    room = torch.zeros(B, m, n + 3, dtype=torch.bfloat16, device="cuda")
    for out in (None, room[:, :, 1:1 + n]):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = rlk.orthogonalise(g, steps=2, coefficients=abc, out=out, status_word=word)
        assert word.item() == rlk.STATUS_NONFINITE and not torch.isfinite(got[1]).all()
        assert torch.equal(got[::2], want[::2])
