"""Layers whose element offsets pass 32 bits: the last rows have the bits of a
call on them alone, or, with whole numbers, the exact result."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
T, H = 528_001, 4096   # 2.16 G elements
TAIL = 1001


def big(seed, H=H):
    """Whole numbers of -3..3."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, (T, H), generator=g, device="cuda", dtype=torch.int8).to(BF)


def test_norm_and_checkpoint(cuda_lib):
    x, dy = big(1), big(2)
    w, b = torch.linspace(0.5, 1.5, H, device="cuda"), torch.linspace(-1, 1, H, device="cuda")
    ck = cuda_lib.new_checkpoint(T, H, x.device)
    y, m, r = cuda_lib.norm(x, w, b, kind=cuda_lib.NORM_LAYER, checkpoint=ck)
    one = cuda_lib.norm(x[-TAIL:], w, b, kind=cuda_lib.NORM_LAYER)
    assert torch.equal(y[-TAIL:], one[0]) and torch.equal(m[-TAIL:], one[1]) and torch.equal(r[-TAIL:], one[2])
    del y
    dx, dw, db = cuda_lib.norm_backward(dy, ck, w, m, r, kind=cuda_lib.NORM_LAYER)
    alone = cuda_lib.checkpoint_pack(x[-TAIL:])
    one = cuda_lib.norm_backward(dy[-TAIL:], alone, w, m[-TAIL:], r[-TAIL:], kind=cuda_lib.NORM_LAYER)
    assert torch.equal(dx[-TAIL:], one[0])
    assert torch.equal(db, dy.sum(0, dtype=torch.float64).float())   # whole numbers below 2^24
    back = cuda_lib.checkpoint_unpack(ck, dtype=BF)
    assert torch.equal(back[-TAIL:], cuda_lib.checkpoint_unpack(alone, dtype=BF))


@pytest.mark.parametrize("K", [64, 65])
def test_linear(cuda_lib, K):
    x, dy = big(3, K), big(4)
    w = torch.randint(-2, 3, (H, K), device="cuda").to(BF)
    y = cuda_lib.linear(x, w, out_dtype=BF)
    for s in (slice(0, TAIL), slice(T - TAIL, T)):
        assert torch.equal(y[s], (x[s].float() @ w.float().T).to(BF))
    del y
    dx, dw, db = cuda_lib.linear_backward(dy, x, w)
    assert torch.equal(dx[-TAIL:], (dy[-TAIL:].double() @ w.double()).to(BF))
    assert torch.equal(dw.double(), dy.T.double() @ x.double())   # below 2^24: exact in fp32
    assert torch.equal(db.double(), dy.sum(0, dtype=torch.float64))
