"""Calls of a distillation step's operators, and of the linear layer, on several streams at once: kernels that take
tensor memory and clusters share the SMs, and every result has the bits that it has alone."""
import pytest
import torch

from _layers import randn
from test_token_logprobs_gpu import given, logits, odd_layout

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def calls(rlk):
    z = odd_layout(logits(400, 20011, BF16, 1))
    ids = given(400, 20011, 3, 1)
    x, wg, wu, dy = randn((300, 520), 1, BF16), randn((700, 520), 2, BF16, 0.05), randn((700, 520), 3, BF16, 0.05), randn((300, 700), 4, BF16)
    big, wbg, wbu = randn((3000, 512), 5, BF16), randn((1500, 512), 6, BF16, 0.05), randn((1500, 512), 7, BF16, 0.05)
    _, gate, up = rlk.gated_linear(x, wg, wu, return_preact=True)
    small, stack, one, large = randn((150, 60, 70), 8), randn((20, 120, 1000), 9), randn((500, 900), 10), randn((6, 1024, 1024), 11, BF16)
    return [lambda: (rlk.orthogonalise(small),), lambda: (rlk.orthogonalise(stack),), lambda: (rlk.orthogonalise(one),), lambda: (rlk.orthogonalise(large),),
            lambda: rlk.gated_linear(big, wbg, wbu, return_preact=True), lambda: (rlk.gated_linear(x[:3], wg, wu),), lambda: (rlk.linear(big, wbg),),
            lambda: rlk.gated_linear_backward(dy, x, wg, wu, gate, up), lambda: rlk.token_logprobs(z, ids, 0.9, n_top=20)]


def test_on_many_streams(cuda_lib):
    work = calls(cuda_lib)
    want = [f() for f in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = [[] for _ in work]
    for turn in range(12):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(work[(k + turn) % len(work)]())
    torch.cuda.synchronize()
    for k in range(len(work)):
        for turn, result in enumerate(got[k]):
            for a, b in zip(result, want[(k + turn) % len(work)]):
                assert torch.equal(a, b), (k, turn)


def test_two_graphs_of_one_workspace(cuda_lib):
    """Replays on one stream, one after the other, also where both graphs use the same workspace."""
    rlk = cuda_lib
    a, b = randn((3, 300, 520), 1), randn((3, 300, 520), 2)
    want = rlk.orthogonalise(a), rlk.orthogonalise(b)
    room = torch.empty(rlk.workspace_size(rlk.OP_ORTHOGONALISE, 3, 300, 520), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty(3, 300, 520, dtype=BF16, device="cuda") for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    for x, out, graph in zip((a, b), outs, graphs):
        with torch.cuda.graph(graph):
            rlk.orthogonalise(x, out=out, workspace=room)
    for _ in range(5):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
