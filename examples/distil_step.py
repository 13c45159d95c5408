"""A distillation step on the library's operators: a student's gated feed-forward
block and head learn a teacher's distribution from its top alternatives.

    teacher's logits -> top alternatives and their log-probabilities
    x -> gated linear -> linear (residual) -> RMS norm -> head -> log-probabilities of those tokens
      -> their backward -> head, norm, linear, gated linear backward -> orthogonalised updates

Random weights and a random teacher; prints the loss and the entropy of each step.

    python examples/distil_step.py [--tokens 2048] [--hidden 512] [--inner 1408] [--vocab 32000] [--top 32] [--steps 8]
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch

import entropy_logits_bf16_gb300 as rlk

BF16 = torch.bfloat16


class Student:
    """The trained weights (fp32 masters, cast to bf16 for the products) and their momenta."""

    def __init__(self, hidden, inner, vocab, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, device=device, generator=g)
        self.w_in = randn(2, inner, hidden) * hidden ** -0.5       # gate, up
        self.w_out = randn(hidden, inner) * inner ** -0.5
        self.gain = torch.ones(hidden, device=device)
        self.w_vocab = randn(vocab, hidden) * 2.0 * hidden ** -0.5
        self.momentum = {name: torch.zeros_like(getattr(self, name)) for name in ("w_in", "w_out")}

    def cast(self):
        return self.w_in.to(BF16), self.w_out.to(BF16), self.w_vocab.to(BF16)


def make_batch(tokens, hidden, vocab, top, seed=1, device="cuda"):
    """Activations, and what is kept of a teacher's rows: its top alternatives with their shares
    of their sum."""
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(tokens, hidden, device=device, generator=g).to(BF16)
    logits = (3.0 * torch.randn(tokens, vocab, device=device, generator=g)).to(BF16)
    _, _, ids, logp = rlk.token_logprobs(logits, None, 1.0, n_top=top)
    return {"x": x, "ids": ids, "share": torch.softmax(logp, 1)}


def gradients(student, batch, entropy_weight=0.0):
    """(loss, mean entropy, {weight: gradient, "x": gradient}): the loss is the mean over the tokens
    of -sum_k share_k ln p(id_k) - entropy_weight H."""
    x, ids = batch["x"], batch["ids"]
    w_in, w_out, w_vocab = student.cast()
    T = x.shape[0]
    y, gate, up = rlk.gated_linear(x, w_in[0], w_in[1], return_preact=True)
    d = rlk.linear(y, w_out, None, x)
    h, _, rstd = rlk.norm(d, student.gain, kind=rlk.NORM_RMS)
    z = rlk.linear(h, w_vocab)
    state = rlk.new_token_state(T, x.device)
    logp, entropy, _, _ = rlk.token_logprobs(z, ids, 1.0, state=state)
    loss = -(batch["share"] * logp).sum() / T - entropy_weight * entropy.mean()
    dz = rlk.token_logprobs_backward(z, ids, 1.0, state, batch["share"] / -T, torch.full_like(entropy, -entropy_weight / T))
    dh, d_vocab, _ = rlk.linear_backward(dz, h, w_vocab, want_bias_grad=False)
    dd, d_gain, _ = rlk.norm_backward(dh, d, student.gain, None, rstd, kind=rlk.NORM_RMS, want_bias_grad=False)
    dy, d_out, _ = rlk.linear_backward(dd, y, w_out, want_bias_grad=False)
    d_in = torch.empty_like(student.w_in)
    dx, _, _, _, _ = rlk.gated_linear_backward(dy, x, w_in[0], w_in[1], gate, up, want_bias_grad=False, grad_w_gate=d_in[0], grad_w_up=d_in[1])
    return loss, entropy.mean(), {"w_in": d_in, "w_out": d_out, "gain": d_gain, "w_vocab": d_vocab, "x": dx + dd}   # the residual's gradient is dd


def step(student, batch, lr=0.02, momentum=0.9, entropy_weight=0.0):
    loss, entropy, grads = gradients(student, batch, entropy_weight)
    for name, m in student.momentum.items():
        m.mul_(momentum).add_(grads[name])
        w = getattr(student, name)
        scale = max(1.0, w.shape[-2] / w.shape[-1]) ** 0.5
        w.add_(rlk.orthogonalise(m), alpha=-lr * scale)             # gate and up: one stack
    for name in ("gain", "w_vocab"):
        getattr(student, name).add_(grads[name], alpha=-lr)
    return loss, entropy


def main():
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("hidden", 512), ("inner", 1408), ("vocab", 32000), ("top", 32), ("steps", 8)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    student, batch = Student(a.hidden, a.inner, a.vocab), make_batch(a.tokens, a.hidden, a.vocab, a.top)
    for k in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        loss, entropy = step(student, batch)
        torch.cuda.synchronize()
        print(f"step {k}: loss {loss.item():.5f}  entropy {entropy.item():.4f}  ({(time.perf_counter() - t) * 1e3:.2f} ms)")


if __name__ == "__main__":
    main()
