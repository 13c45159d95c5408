"""The pairs' epilogue with two columns a lane: an even N and rows of y, z or the
residual on 4-byte but not on 16-byte boundaries, in tiles enough for pairs of CTAs.
Whole numbers that bf16 holds, so every output is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ints(shape, top, seed, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(dtype)


def inside(t, ld, first):
    """A view of t's shape in rows of ld elements, from column `first` on, and its buffer of NaN."""
    buf = torch.full((t.shape[0] + 1, ld), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[:-1, first:first + t.shape[1]]
    return view, buf


# more than 152 tiles of 128 x 128, a ragged last row and column of tiles of 256 x 256
@pytest.mark.parametrize("M,N", [(1531, 2050), (1300, 2308), (5003, 770)])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("act", [0, 3])
@pytest.mark.parametrize("bias,res", [(F32, True), (BF, False), (None, True)])
def test_rows_on_four_bytes(cuda_lib, M, N, out, act, bias, res):
    K = 72
    x, w = ints((M, K), 1, 1), ints((N, K), 1, 2)
    b = None if bias is None else ints((N,), 9, 3, bias)
    r = ints((M, N), 40, 4) if res else None
    if res:   # rows of N + 6 elements from the second on: 4 bytes off 16
        held, _ = inside(r, (N + 6) // 4 * 4 + 2, 2)
        held.copy_(r)
        assert held.data_ptr() % 16 == 4 and held.stride(0) % 8 in (2, 6)
    y, buf = inside(torch.empty((M, N), dtype=out, device="cuda"), (N + 9) // 4 * 4 + 2, 2)
    got, z = cuda_lib.linear(x, w, b, held if res else None, activation=act, return_preact=True, out=y)
    want = x.double() @ w.double().t() + (0 if b is None else b.double())
    assert torch.equal(z.double(), want)
    want = (want.clamp_min(0) if act else want) + (r.double() if res else 0)
    assert torch.equal(got.double(), want)
    y.fill_(float("nan"))
    assert bool(torch.isnan(buf).all())   # nothing beside the rows


@pytest.mark.parametrize("M,N", [(1531, 2050), (1300, 2308)])
def test_residual_in_place(cuda_lib, M, N):
    x, w, r = ints((M, 72), 1, 5), ints((N, 72), 1, 6), ints((M, N), 40, 7)
    y = r.clone()
    assert y.data_ptr() % 16 == 0 and N % 8
    cuda_lib.linear(x, w, None, y, out=y)
    assert torch.equal(y.double(), x.double() @ w.double().t() + r.double())


def test_gradients(cuda_lib):
    """dx and dw [., 2050] and [., 2306] as their products leave them."""
    M, N, K = 1531, 2050, 2306
    dy, x, w = ints((M, N), 1, 8), ints((M, K), 1, 9), ints((N, K), 1, 10)
    dx, dw, db = cuda_lib.linear_backward(dy, x, w, grad_dtype=F32)
    assert torch.equal(dx.double(), dy.double() @ w.double()) and torch.equal(dw.double(), dy.double().t() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))
    dx, dw, _ = cuda_lib.linear_backward(dy, x, w, weight_grad_dtype=BF)
    assert torch.equal(dx.double(), (dy.double() @ w.double()).to(BF).double())
    assert torch.equal(dw.double(), (dy.double().t() @ x.double()).to(BF).double())
