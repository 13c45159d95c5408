"""Stacks of small matrices on both sides of the limits up to which one kernel takes them."""
import pytest
import torch

from _layers import randn
from test_orthogonalise_gpu import check, orth64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(91, 128, 384), (92, 128, 384), (68, 64, 512), (69, 64, 512), (76, 512, 64), (45, 128, 768), (46, 768, 128), (29, 128, 896), (30, 128, 896), (26, 1024, 128),
                                   (27, 128, 1024), (12, 64, 1024), (13, 64, 1024), (14, 896, 64), (15, 896, 64)], ids=str)
def test_by_the_number_of_matrices(cuda_lib, shape):
    g = randn(shape, 3, torch.bfloat16)
    got = cuda_lib.orthogonalise(g)
    check(got, orth64(g))
    assert torch.equal(cuda_lib.orthogonalise(g), got)
