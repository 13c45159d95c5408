"""Workspaces of a distillation step's operators: whatever they hold on entry (0xFF bytes are NaN in fp16, bf16 and
fp32), the result has the same bits, and nothing is written behind the size that rlk_workspace_size gives."""
import pytest
import torch

from _layers import randn
from test_gated_gpu import laid_out

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 1 << 16


def with_workspaces(need, call, plain):
    """`call(workspace)` with workspaces of zeros, of NaN and of what a call left; each result's bits against `plain`'s."""
    room = torch.empty(need + GUARD, dtype=torch.uint8, device="cuda")
    for fill in (0x00, 0xFF, None):
        if fill is not None:
            room[:need] = fill
        room[need:] = 0x5A
        got = call(room[:need])
        for a, b in zip(got, plain):
            assert (a is None) == (b is None)
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)), fill
        assert (room[need:] == 0x5A).all()


# one kernel with one and several CTAs; launches: numbers in two halves, all of A's tiles, its blocks of 128, of 256
# by single CTAs and by pairs, X's tiles by pairs; stacks; sides off 8 and 16
SHAPES = [(1, 64, 64), (3, 120, 1000), (3, 1000, 120), (2, 7, 5), (1, 100, 1101), (1, 1101, 100), (30, 128, 1024), (1, 501, 500), (1, 300, 703), (1, 703, 300), (1, 951, 1301),
          (1, 1301, 951), (1, 900, 3000), (1, 900, 5000), (1, 5000, 900), (1, 2600, 2201), (1, 2201, 2600), (24, 131, 203), (6, 1024, 1024), (30, 403, 300), (24, 512, 1024)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_orthogonalise(cuda_lib, shape, dtype):
    rlk = cuda_lib
    g = randn(shape, 1, dtype)
    need = rlk.workspace_size(rlk.OP_ORTHOGONALISE, *shape)
    plain = rlk.orthogonalise(g)
    assert torch.isfinite(plain).all()
    with_workspaces(need, lambda ws: (rlk.orthogonalise(g, workspace=ws),), (plain,))


SIZES = [(5, 70, 201), (17, 1001, 7), (64, 257, 1001), (129, 643, 1025), (300, 130, 4097), (521, 1301, 1003), (2500, 1401, 193), (8, 64, 128)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("odd", [False, True, "even"])
def test_gated_linear(cuda_lib, M, N, K, odd):
    rlk = cuda_lib
    x, wg, wu = (laid_out(t, odd) for t in (randn((M, K), 1, BF), randn((N, K), 2, BF, K ** -0.5), randn((N, K), 3, BF, K ** -0.5)))
    need = rlk.workspace_size(rlk.OP_GATED_LINEAR, M, N, K)
    plain = rlk.gated_linear(x, wg, wu, return_preact=True)
    assert all(torch.isfinite(t).all() for t in plain)
    with_workspaces(need, lambda ws: rlk.gated_linear(x, wg, wu, return_preact=True, workspace=ws), plain)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("odd", [False, True, "even", "checkpoint"])
def test_gated_linear_backward(cuda_lib, M, N, K, odd):
    rlk = cuda_lib
    lay = lambda t: laid_out(t, odd if odd != "checkpoint" else False)
    x = randn((M, K), 5, BF)
    kept = rlk.checkpoint_pack(x) if odd == "checkpoint" else lay(x)
    wg, wu = lay(randn((N, K), 6, BF, K ** -0.5)), lay(randn((N, K), 7, BF, K ** -0.5))
    gate, up, dy = lay(randn((M, N), 8, BF)), lay(randn((M, N), 9, BF)), lay(randn((M, N), 10, BF, 0.1))
    need = rlk.workspace_size(rlk.OP_GATED_LINEAR_BWD, M, N, K)
    for wants in (dict(), dict(want_weight_grad=False), dict(want_x_grad=False, want_bias_grad=False), dict(want_x_grad=False, want_weight_grad=False)):
        plain = rlk.gated_linear_backward(dy, kept, wg, wu, gate, up, **wants)
        assert all(t is None or torch.isfinite(t).all() for t in plain)
        with_workspaces(need, lambda ws: rlk.gated_linear_backward(dy, kept, wg, wu, gate, up, workspace=ws, **wants), plain)
