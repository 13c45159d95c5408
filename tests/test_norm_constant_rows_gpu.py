"""Layer norm of rows that hold one value (or none but it): every sum of them is exact, so
the mean is that value, the deviations are 0 and y is the bias, whatever the width."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
VALUES = [0.0, 1.0, -7.0, 3.140625, 100.0, -1000.0, 29952.0]   # 8 bits: times a width below 2^16, exact in fp32


# widths on chip (16 and 32 columns a thread, aligned or not) and wider ones, among them
# such whose fp32 reciprocal times the sum is not the value
@pytest.mark.parametrize("H", [1, 7, 100, 1000, 1001, 3608, 4096, 5003, 5992, 8200, 10689, 10952, 16384, 17000, 21324, 40000])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("eps", [1e-5, 1e-12])
def test_constant_rows(cuda_lib, H, dtype, eps):
    x = torch.tensor(VALUES, device="cuda")[:, None].expand(-1, H).to(dtype).contiguous()
    b = torch.linspace(-2, 2, H, device="cuda")
    y, mean, rstd = cuda_lib.norm(x, torch.full((H,), 3.0, device="cuda"), b, eps=eps)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, b.to(dtype).expand(len(VALUES), H))
    want = torch.full_like(rstd, eps).double().rsqrt()
    assert bool(((rstd.double() - want).abs() <= 4 * 2.0 ** -24 * want).all())
