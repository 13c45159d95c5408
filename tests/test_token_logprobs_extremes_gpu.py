"""Temperatures and logits near the ends of fp32's range against 64 bits."""
import pytest
import torch

from test_token_logprobs_gpu import given, odd_layout

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# short rows; a few rows shared by CTAs; whole rows a CTA; the ring (many long rows off 16 bytes)
@pytest.mark.parametrize("T,V", [(3, 3000), (2, 70001), (60, 20011), (320, 20011)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("temp,size", [(3e37, 1e33), (3.2e37, 1e33), (3.2e37, 7e37), (3e38, 1e35), (3e38, 7e37), (1e36, 7e37), (4e36, 7e37)])
def test_high_temperatures(cuda_lib, T, V, dtype, temp, size):
    """Logits up to 2 `size` in magnitude (their distances below 3.4e38), exponents up to 280."""
    rlk, keep = cuda_lib, torch.arange(0, T, max(1, T // 3))
    g = torch.Generator().manual_seed(V)
    z = (torch.randn(T, V, generator=g).clamp(-2, 2).double() * size).to(dtype).cuda()
    z = odd_layout(z) if T > 2 else z
    ids = given(T, V, 3, 1)
    state = rlk.new_token_state(T, "cuda")
    lp, h, ti, tl = rlk.token_logprobs(z, ids, temp, n_top=3, state=state)
    temp32 = torch.tensor(temp, dtype=F32).double().item()            # as the call takes it
    x = z[keep].double().cpu() / temp32
    want = torch.log_softmax(x, 1)
    p = want.exp()
    H = -(p * want).sum(1)
    # d = (z - M) / T to three roundings of it, on the average H + ln V at most; S to V / 1024 + 50 of them
    e, ln = 2 ** -24, torch.log(torch.tensor(float(V))).item() + 1
    S = (V / 1024 + 50 + 4 * (H + ln)) * e
    assert ((h[keep].double().cpu() - H).abs() <= S + (2 * (V / 1024 + 50) * (H + ln) + 8 * (H + ln) ** 2 + 3 * ln) * e).all()
    for got, i in ((lp, ids), (tl, ti)):
        i = i[keep].cpu().long()
        ref = torch.gather(want, 1, i.clamp_min(0)).masked_fill(i < 0, 0.0)
        d = torch.gather(x.max(1, keepdim=True)[0] - x, 1, i.clamp_min(0))
        assert ((got[keep].double().cpu() - ref).abs() <= S[:, None] + (4 * d + 3 * ln + 2 * ref.abs()) * e).all()
    assert torch.equal(z[keep].gather(1, ti[keep].long()).float(), z[keep].float().topk(3, 1)[0])
    dz = rlk.token_logprobs_backward(z, ids, temp, state, torch.ones_like(lp), grad_dtype=F32)
    n = (ids[keep] >= 0).sum(1, keepdim=True).cpu()
    named = torch.zeros(len(keep), V + 1, dtype=torch.float64)
    i = ids[keep].cpu().long()
    named.scatter_add_(1, torch.where(i < 0, V, i), torch.ones_like(i, dtype=torch.float64))
    ref = (named[:, :V] - n * p) / temp32
    # p's relative error as S's and the exponent's (d at most 280); below 2^-126 fp32 has 2^-149 steps, here also flushed
    err = (dz[keep].double().cpu() - ref).abs()
    assert (err <= (named[:, :V] + n * p) / temp32 * (V / 1024 + 60 + 4 * 280) * e + 2.0 ** -126).all()
