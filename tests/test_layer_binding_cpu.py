"""The layers' binding on the host: what it refuses before the library is called.
Tensors that say that they are on a CUDA device stand in for such ones; launches are
made to fail."""
import pytest
import torch

import entropy_logits_bf16_gb300 as rlk

BF, F32 = torch.bfloat16, torch.float32


class OnCuda(torch.Tensor):
    is_cuda = property(lambda self: True)


def cuda(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnCuda)


@pytest.fixture(autouse=True)
def lib(monkeypatch):
    rlk.build()
    lib = rlk.load()
    monkeypatch.setattr(rlk, "_stream", lambda device: 0)
    lib.rlk_debug_inject_launch_failures(1000)
    yield lib
    lib.rlk_debug_inject_launch_failures(0)


def test_workspaces_on_the_host_are_refused():
    dy, x, w, r = cuda(4, 64), cuda(4, 64), cuda(64), cuda(4)
    off, lp = cuda(5, dtype=torch.int32), cuda(50)
    for call in (lambda ws: rlk.norm_backward(dy, x, w, None, r, kind=rlk.NORM_RMS, workspace=ws),
                 lambda ws: rlk.preference_loss(lp, None, off, workspace=ws)):
        with pytest.raises(rlk.RlkError):      # on the device: on to the launch, which fails
            call(cuda(1 << 16, dtype=torch.uint8))
        with pytest.raises(ValueError):
            call(torch.zeros(1 << 16, dtype=torch.uint8))


def test_a_checkpoint_follows_its_tensors(lib, monkeypatch):
    """Replaced tensors are the ones that the entry points get, whatever was there before."""
    T, H = 4, 100
    ck = rlk.Checkpoint(cuda(T, 112, dtype=torch.int8), cuda(T, 16, dtype=torch.uint8), T, H)
    seen = []
    monkeypatch.setattr(lib, "rlk_checkpoint_unpack", lambda c, *rest: seen.append(
        (c._obj.codes, c._obj.scales, c._obj.ld_codes, c._obj.ld_scales)) or 0)
    out = cuda(T, H)
    rlk.checkpoint_unpack(ck, out=out)
    first = ck.codes, ck.scales
    ck.codes, ck.scales = cuda(T, 128, dtype=torch.int8), cuda(T, 4, dtype=torch.uint8)
    rlk.checkpoint_unpack(ck, out=out)
    assert seen == [(first[0].data_ptr(), first[1].data_ptr(), 112, 16), (ck.codes.data_ptr(), ck.scales.data_ptr(), 128, 4)]
    good = ck.codes
    for bad in (torch.zeros(T, 112, dtype=torch.int8), cuda(T, 112, dtype=torch.uint8), cuda(T, 96, dtype=torch.int8),
                cuda(T + 1, 112, dtype=torch.int8), cuda(T, 224, dtype=torch.int8)[:, ::2]):
        ck.codes = bad
        with pytest.raises(ValueError):
            rlk.checkpoint_unpack(ck, out=out)
        with pytest.raises(ValueError):
            rlk.Checkpoint(bad, ck.scales, T, H)
    ck.codes, ck.scales = good, cuda(T, 3, dtype=torch.uint8)
    with pytest.raises(ValueError):
        rlk.checkpoint_unpack(ck, out=out)


def plain_norm(x, w, b, **kw):
    r = (x * x).mean(1).rsqrt()
    return x * r[:, None] * w, None, r


def plain_calls(monkeypatch):
    """Plain forms in place of the library's calls."""
    monkeypatch.setattr(rlk, "norm", plain_norm)
    monkeypatch.setattr(rlk, "norm_backward", lambda dy, x, w, m, r, **kw: (dy * w * r[:, None], (dy * x).sum(0), None))
    monkeypatch.setattr(rlk, "linear", lambda x, w, b, r, **kw: (x @ w.t(), x @ w.t()) if kw else x @ w.t())
    monkeypatch.setattr(rlk, "linear_backward", lambda dy, x, w, z, **kw: (dy @ w, dy.t() @ x, None))
    monkeypatch.setattr(rlk, "logprob_entropy", lambda x, ids, *a, **kw: (x.sum(1), x.square().sum(1)))
    monkeypatch.setattr(rlk, "logprob_entropy_backward", lambda x, ids, t, state, g, h: g[:, None] + 2 * x)


@pytest.mark.parametrize("op", ["norm", "linear", "logprob"])
def test_second_derivatives_are_refused(monkeypatch, op):
    """The gradients are the library's numbers: autograd cannot go through them, and
    says so instead of taking them for constants."""
    plain_calls(monkeypatch)
    x, w = torch.randn(4, 8, requires_grad=True), torch.randn(8, requires_grad=True)
    if op == "norm":
        y = rlk.norm_autograd(x, w, kind=rlk.NORM_RMS)
    elif op == "linear":
        y = rlk.linear_autograd(x, torch.randn(6, 8, requires_grad=True), activation=rlk.ACT_GELU)
    else:
        y = sum(rlk.logprob_entropy_autograd(x, torch.zeros(4, dtype=torch.int32), 1.0, 1.0))
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|differentiate twice"):
        (g.sum() + x.sum()).backward()


def test_output_types_are_refused_like_inputs():
    x, w = cuda(4, 64, dtype=BF), cuda(32, 64, dtype=BF)
    for call in (lambda: rlk.norm(x, out_dtype=torch.float16), lambda: rlk.linear(x, w, out_dtype=torch.float64),
                 lambda: rlk.linear_backward(cuda(4, 32, dtype=BF), x, w, grad_dtype=torch.float16),
                 lambda: rlk.norm_backward(x, x, None, None, cuda(4), kind=rlk.NORM_RMS, grad_dtype=torch.float16),
                 lambda: rlk.checkpoint_unpack(rlk.Checkpoint(cuda(4, 64, dtype=torch.int8), cuda(4, 2, dtype=torch.uint8), 4, 64),
                                               out=cuda(4, 64, dtype=torch.float16))):
        with pytest.raises(ValueError):
            call()


def laid_out(rows, cols, how):
    """bf16 rows that start on 16-byte boundaries, or whose stride or base is off them."""
    if how == "aligned":
        return cuda(rows, cols + 8 - cols % 8, dtype=BF)[:, :cols]
    return cuda(rows, cols + 1, dtype=BF)[:, :cols] if how == "stride" else cuda(rows, cols + 16 - cols % 8, dtype=BF)[:, 3:3 + cols]


def exactly(real, seen):
    """The entry point with the workspace given, and with a byte less."""
    def call(*a):
        *head, ws, size, stream = a
        seen.append(size)
        if size:
            assert real(*head, ws, size - 1, stream) == 3
        return real(*a)
    return call


@pytest.mark.parametrize("M", [1, 4, 5, 33])
@pytest.mark.parametrize("N,K", [(96, 130), (31, 64)])
@pytest.mark.parametrize("x_how", ["aligned", "stride", "base"])
@pytest.mark.parametrize("w_how", ["aligned", "stride", "base"])
def test_linear_asks_for_the_workspace_that_it_uses(lib, monkeypatch, M, N, K, x_how, w_how):
    seen = []
    monkeypatch.setattr(lib, "rlk_linear_fwd", exactly(lib.rlk_linear_fwd, seen))
    monkeypatch.setattr(lib, "rlk_linear_bwd", exactly(lib.rlk_linear_bwd, seen))
    x, w = laid_out(M, K, x_how), laid_out(N, K, w_how)
    with pytest.raises(rlk.RlkError) as e:
        rlk.linear(x, w)
    assert e.value.code == 4 and (seen[-1] > 0) == (M > 4 and (x_how, w_how) != ("aligned", "aligned"))
    kept = rlk.Checkpoint(cuda(M, -(-K // 16) * 16, dtype=torch.int8), cuda(M, 16, dtype=torch.uint8), M, K)
    for act in (rlk.ACT_NONE, rlk.ACT_GELU):
        for dy_how in ("aligned", "stride"):
            for wants in range(1, 8):
                for src in (x, kept):
                    dy, z = laid_out(M, N, dy_how), cuda(M, N, dtype=BF) if act else None
                    with pytest.raises(rlk.RlkError) as e:
                        rlk.linear_backward(dy, src, w, z, activation=act, want_x_grad=bool(wants & 1),
                                            want_weight_grad=bool(wants & 2), want_bias_grad=bool(wants & 4))
                    assert e.value.code == 4
