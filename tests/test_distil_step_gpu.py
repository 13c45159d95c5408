"""The operators of a distillation step together, as examples/distil_step.py runs them: the
step's gradients against a 64-bit autograd of the same model, its updates against the
operators' own results, and the whole of it captured into a graph.

Tolerance of a gradient, as a ratio of 2-norms: between the loss and a weight lie roundings to
bf16 (at most 2^-8 of a value, 0.0023 of a tensor in the root mean square) of y, the block's
output, h, the logits and of five gradients, and of dg and du; that of the logits moves
the probabilities by 0.0023 of |z|, about 2 here.  In quadrature 10 x 0.0023^2 + (2 x 0.0023)^2:
0.0086; a tensor's later ones act through sums that keep the ratio.  Twice that is held.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference(student, batch, entropy_weight):
    """The model in 64 bits on the same bf16 weights."""
    x = batch["x"].double().requires_grad_()
    w_in, w_out, w_vocab = (t.double().requires_grad_() for t in student.cast())
    gain = student.gain.double().requires_grad_()
    d = (torch.nn.functional.silu(x @ w_in[0].t()) * (x @ w_in[1].t())) @ w_out.t() + x
    h = d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt() * gain
    logp = torch.log_softmax(h @ w_vocab.t(), 1)
    entropy = -(logp.exp() * logp).sum(1).mean()
    loss = -(batch["share"].double() * logp.gather(1, batch["ids"].long())).sum(1).mean() - entropy_weight * entropy
    loss.backward()
    return loss, entropy, dict(x=x.grad, w_in=w_in.grad, w_out=w_out.grad, gain=gain.grad, w_vocab=w_vocab.grad)


@pytest.mark.parametrize("tokens,hidden,inner,vocab,top", [(37, 128, 200, 1000, 8), (300, 320, 501, 4001, 64), (700, 200, 352, 2048, 1)])
def test_gradients_of_the_step(cuda_lib, tokens, hidden, inner, vocab, top):
    import distil_step as ds
    student, batch = ds.Student(hidden, inner, vocab, seed=3), ds.make_batch(tokens, hidden, vocab, top, seed=4)
    loss, entropy, grads = ds.gradients(student, batch, 0.1)
    want, want_entropy, refs = reference(student, batch, 0.1)
    assert abs(loss.item() - want.item()) <= 0.01 and abs(entropy.item() - want_entropy.item()) <= 0.01
    for name, g in grads.items():
        r = refs[name]
        assert ((g.double() - r).norm() / r.norm()).item() <= 0.0172, name


def test_the_updates(cuda_lib):
    """A step moves each matrix by its orthogonalised momentum, a stack as its matrices one by one."""
    import distil_step as ds
    student, batch = ds.Student(192, 264, 1500), ds.make_batch(256, 192, 1500, 16)
    before = {n: getattr(student, n).clone() for n in ("w_in", "w_out", "gain", "w_vocab")}
    _, _, grads = ds.gradients(student, batch)
    ds.step(student, batch, lr=0.02)
    for name in ("w_in", "w_out"):
        g = grads[name]
        update = torch.stack([cuda_lib.orthogonalise(m) for m in g]) if g.dim() == 3 else cuda_lib.orthogonalise(g)
        scale = max(1.0, g.shape[-2] / g.shape[-1]) ** 0.5
        moved = (before[name] - getattr(student, name)) / (0.02 * scale)
        # one matrix and a stack of two may split their sums differently: a bf16 rounding apart; the difference
        # of two fp32 weights of up to 0.5 keeps 2^-25 / 0.02 of it
        assert ((moved - update.float()).abs() <= 2 ** -7 * update.float().abs() + 1e-4).all()
        s = torch.linalg.svdvals(moved.double())
        assert s.max() < 1.3
    for name in ("gain", "w_vocab"):
        assert torch.equal(getattr(student, name), before[name].add(grads[name], alpha=-0.02))


def test_the_step_in_a_graph(cuda_lib):
    import distil_step as ds
    student, batch = ds.Student(128, 200, 2000), ds.make_batch(64, 128, 2000, 8)
    run = lambda: ds.gradients(student, batch, 0.01)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, entropy, grads = run()
        updates = [cuda_lib.orthogonalise(grads[n]) for n in ("w_in", "w_out")]
    batch["x"].copy_(ds.make_batch(64, 128, 2000, 8, seed=9)["x"])
    student.w_in.mul_(0.9)
    graph.replay()
    torch.cuda.synchronize()
    want_loss, want_entropy, want = run()
    assert torch.equal(loss, want_loss) and torch.equal(entropy, want_entropy)
    assert all(torch.equal(grads[n], want[n]) for n in grads)
    assert all(torch.equal(u, cuda_lib.orthogonalise(want[n])) for u, n in zip(updates, ("w_in", "w_out")))


def test_the_example_runs(cuda_lib):
    import distil_step as ds
    student, batch = ds.Student(64, 96, 500), ds.make_batch(40, 64, 500, 4)
    for _ in range(2):
        loss, entropy = ds.step(student, batch)
        assert torch.isfinite(loss) and torch.isfinite(entropy)


def test_autograd_forms_together(cuda_lib):
    """The same gradients through the differentiable forms."""
    import distil_step as ds
    rlk = cuda_lib
    student, batch = ds.Student(96, 160, 700), ds.make_batch(50, 96, 700, 5)
    _, _, grads = ds.gradients(student, batch, 0.1)
    w_in, w_out, w_vocab = (t.requires_grad_() for t in student.cast())
    x = batch["x"].clone().requires_grad_()
    y = rlk.gated_linear_autograd(x, w_in[0], w_in[1])
    h = rlk.norm_autograd(rlk.linear_autograd(y, w_out, None, x), student.gain, kind=rlk.NORM_RMS)
    logp, entropy, _, _ = rlk.token_logprobs_autograd(rlk.linear_autograd(h, w_vocab), batch["ids"])
    (-(batch["share"] * logp).sum(1).mean() - 0.1 * entropy.mean()).backward()
    for name, t in (("w_in", w_in), ("w_out", w_out), ("w_vocab", w_vocab), ("x", x)):
        # the weights' gradients rounded to bf16 here; x's is added up in another order
        assert ((t.grad.float() - grads[name].float()).norm() <= 0.006 * grads[name].float().norm()), name
