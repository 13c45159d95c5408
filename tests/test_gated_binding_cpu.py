"""The gated layer's binding on the host: one tensor for both gradients is refused (its two products would
be added up in no order).  Tensors that say that they are on a CUDA device stand in for such ones; launches
are made to fail."""
import pytest
import torch

import entropy_logits_bf16_gb300 as rlk
from test_layer_binding_cpu import cuda, lib  # noqa: F401

BF = torch.bfloat16


@pytest.mark.parametrize("accumulate", [False, True])
def test_one_tensor_for_both_gradients(accumulate):
    dy, x, w = cuda(4, 8, dtype=BF), cuda(4, 16, dtype=BF), cuda(8, 16, dtype=BF)
    call = lambda dwg, dwu, dbg, dbu: rlk.gated_linear_backward(dy, x, w, w, dy, dy, grad_w_gate=dwg, grad_w_up=dwu, grad_bias_gate=dbg,
                                                                grad_bias_up=dbu, accumulate=accumulate)
    both, wide, biases = cuda(2, 8, 16), cuda(8, 32), cuda(2, 8)
    for bad in ((both[0], both[0], biases[0], biases[1]), (both[0], both[1], biases[0], biases[0])):
        with pytest.raises(ValueError, match="of their own"):
            call(*bad)
    for good in ((both[0], both[1], biases[0], biases[1]), (wide[:, :16], wide[:, 16:], biases[0], biases[1])):
        with pytest.raises(rlk.RlkError):      # on to the launch, which fails
            call(*good)
