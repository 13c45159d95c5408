"""The gradient of the token log-probabilities in every pair of types and layouts: a row's bits do not depend on where
it starts, on 2, 4, 8 or 16 bytes, and nothing beside it is written.  (Values: test_token_logprobs_gpu.)"""
import pytest
import torch

from test_token_logprobs_gpu import given, logits, odd_layout

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("V", [3, 12, 1004, 4098, 4099, 20012, 33001])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gdt", [BF16, F32], ids=["to_bf16", "to_f32"])
def test_rows_by_where_they_start(cuda_lib, V, dtype, gdt):
    rlk, T, temp = cuda_lib, 5, 0.8
    z, ids = logits(T, V, dtype, V, "masked" if V > 100 else "peaked"), given(T, V, 4, 1)
    g = torch.Generator().manual_seed(V)
    glp, gh = torch.randn(T, 4, generator=g).cuda(), torch.randn(T, generator=g).cuda()
    state = rlk.new_token_state(T, "cuda")
    rlk.token_logprobs(z, ids, temp, state=state)
    want = None
    for lead_in in range(5):                                           # contiguous, then off 16 bytes by each place
        x = odd_layout(z, lead_in) if lead_in else z
        for pitch in (V, (V + 15) // 8 * 8, (V + 15) // 8 * 8 + 4, V + 9):
            for lead in range(9):
                room = torch.full((T * pitch + 16,), 7.0, dtype=gdt, device="cuda")
                out = room[lead:lead + T * pitch].view(T, pitch)[:, :V]
                rlk.token_logprobs_backward(x, ids, temp, state, glp, gh, out=out)
                want = out.clone() if want is None else want
                assert torch.equal(out, want), (lead_in, pitch, lead)
                out.fill_(7.0)
                assert (room == 7.0).all(), (lead_in, pitch, lead)
    assert torch.isfinite(want).all()
