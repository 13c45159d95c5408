"""The operators together, as examples/preference_step.py runs them: the step's
gradients against a 64-bit autograd of the same model, and training that lowers
the loss.

Tolerance of a gradient, as a ratio of 2-norms: between the loss and a weight lie
roundings to bf16 of y, h, the logits' gradient, dy and dz (2^-9 each, rms 2^-9
/ sqrt 3 of its tensor) and the two 8-bit checkpoints (rms error at most
1 / 127 / sqrt 3 of a block's largest value, about a third of that of its rms
value: 1.5 %).  Added in quadrature: below 2.5 %.
"""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference(head, batch, logp_ref, beta):
    """The model in 64 bits on the same bf16 weights."""
    x = batch["x"].double().requires_grad_()
    w, w_vocab = (t.double().requires_grad_() for t in head.cast())
    b, gain = head.b.double().requires_grad_(), head.gain.double().requires_grad_()
    y = torch.nn.functional.gelu(x @ w.t() + b) + x
    h = y * (y.square().mean(1, keepdim=True) + 1e-5).rsqrt() * gain
    logp = torch.log_softmax(h @ w_vocab.t(), 1).gather(1, batch["ids"].long()[:, None])[:, 0]
    off, m = batch["off"].tolist(), batch["mask"].double()
    d = (logp - logp_ref.double()) * m
    s = torch.stack([d[a:e].sum() for a, e in zip(off, off[1:])])
    loss = -torch.nn.functional.logsigmoid(beta * (s[0::2] - s[1::2])).mean()
    loss.backward()
    return loss, dict(x=x.grad, w=w.grad, b=b.grad, gain=gain.grad, w_vocab=w_vocab.grad)


@pytest.mark.parametrize("hidden,vocab,pairs", [(128, 1000, 3), (320, 4001, 6)])
def test_gradients_of_the_step(cuda_lib, hidden, vocab, pairs):
    import preference_step as ps
    head, batch = ps.Head(hidden, vocab, seed=3), ps.make_batch(pairs, 5, 60, hidden, vocab, seed=4)
    logp, _ = ps.forward(head, batch)
    logp_ref = logp + 0.05 * torch.randn(logp.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    loss, stats, grads = ps.gradients(head, batch, logp_ref, beta=0.3)
    want, refs = reference(head, batch, logp_ref, 0.3)
    assert abs(loss.item() - want.item()) <= 0.01
    for name, g in grads.items():
        r = refs[name]
        assert ((g.double() - r).norm() / r.norm()).item() <= 0.025, name


def test_training_lowers_the_loss(cuda_lib):
    import preference_step as ps
    head, batch = ps.Head(256, 2000), ps.make_batch(8, 10, 80, 256, 2000)
    logp_ref, _ = ps.forward(head, batch)
    losses, margins = [], []
    for _ in range(6):
        loss, stats = ps.step(head, batch, logp_ref)
        losses.append(loss.item())
        margins.append(stats[3].item())
    assert losses[0] == pytest.approx(0.6931, abs=1e-4)          # no preference yet: ln 2
    assert all(b < a for a, b in zip(losses, losses[1:])) and margins[-1] > margins[0]
