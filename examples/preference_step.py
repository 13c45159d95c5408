"""A preference-training step on the library's operators, from the last block's
activations to the weights' update:

    x -> linear (bias, GELU, residual) -> RMS norm -> LM head + scorer -> preference loss
      -> LM head backward -> norm backward -> linear backward -> SGD

The activations that the backward needs (x and the norm's input) are kept as
8-bit checkpoints.  Random weights and responses; prints the loss and the
reward margin of each step.

    python examples/preference_step.py [--pairs 16] [--hidden 1024] [--vocab 32000] [--steps 8]
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch

import entropy_logits_bf16_gb300 as rlk

BF16 = torch.bfloat16


class Head:
    """The trained weights: fp32 masters, cast to bf16 for the products."""

    def __init__(self, hidden, vocab, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, device=device, generator=g)
        self.w = randn(hidden, hidden) * hidden ** -0.5
        self.b = torch.zeros(hidden, device=device)
        self.gain = torch.ones(hidden, device=device)
        self.w_vocab = randn(vocab, hidden) * 0.02

    def cast(self):
        return self.w.to(BF16), self.w_vocab.to(BF16)


def make_batch(pairs, lo, hi, hidden, vocab, seed=1, device="cuda"):
    """Packed responses: sequences 2 i and 2 i + 1 answer one prompt, the first
    preferred.  A tenth of the tokens (the prompts' tails) is masked."""
    g = torch.Generator(device=device).manual_seed(seed)
    lens = torch.randint(lo, hi + 1, (2 * pairs,), device=device, generator=g)
    off = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
    n = int(off[-1])
    return {"x": torch.randn(n, hidden, device=device, generator=g).to(BF16),
            "ids": torch.randint(0, vocab, (n,), device=device, generator=g, dtype=torch.int32),
            "off": off,
            "mask": (torch.rand(n, device=device, generator=g) >= 0.1).to(torch.uint8)}


def forward(head, batch, keep=False):
    """Log-probabilities of the responses' tokens, and what the backward needs."""
    x = batch["x"]
    w, w_vocab = head.cast()
    y, z = rlk.linear(x, w, head.b, x, activation=rlk.ACT_GELU, return_preact=True)
    ck_y = rlk.new_checkpoint(y.shape[0], y.shape[1], y.device) if keep else None
    h, _, rstd = rlk.norm(y, head.gain, kind=rlk.NORM_RMS, checkpoint=ck_y)
    lse = torch.empty(x.shape[0], device=x.device)
    logp, entropy = rlk.lmhead_logprob(h, w_vocab, batch["ids"], 1.0, out_lse=lse)
    if not keep:
        return logp, None
    return logp, dict(w=w, w_vocab=w_vocab, z=z, ck_x=rlk.checkpoint_pack(x), ck_y=ck_y, h=h, rstd=rstd,
                      lse=lse, entropy=entropy)


def gradients(head, batch, logp_ref, beta=0.1):
    """(loss, statistics, {weight: gradient, "x": gradient}) of one batch."""
    logp, s = forward(head, batch, keep=True)
    loss, dlogp, _, stats = rlk.preference_loss(logp, logp_ref, batch["off"], loss_mask=batch["mask"], beta=beta)
    dh, d_vocab = rlk.lmhead_backward(s["h"], s["w_vocab"], batch["ids"], 1.0, s["lse"], s["entropy"],
                                      grad_logprob=dlogp)
    dy, d_gain, _ = rlk.norm_backward(dh, s["ck_y"], head.gain, None, s["rstd"], kind=rlk.NORM_RMS,
                                      grad_dtype=BF16, want_bias_grad=False)
    dx, dw, db = rlk.linear_backward(dy, s["ck_x"], s["w"], s["z"], activation=rlk.ACT_GELU)
    return loss, stats, {"w": dw, "b": db, "gain": d_gain, "w_vocab": d_vocab, "x": dx + dy}   # the residual's gradient is dy


def step(head, batch, logp_ref, lr=1e-3, beta=0.1):
    loss, stats, grads = gradients(head, batch, logp_ref, beta)
    for name in ("w", "b", "gain", "w_vocab"):
        getattr(head, name).add_(grads[name], alpha=-lr)
    return loss, stats


def main():
    p = argparse.ArgumentParser()
    for name, value in (("pairs", 16), ("hidden", 1024), ("vocab", 32000), ("steps", 8)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    head, batch = Head(a.hidden, a.vocab), make_batch(a.pairs, 64, 512, a.hidden, a.vocab)
    logp_ref, _ = forward(head, batch)   # the reference policy: the weights before training
    for k in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        loss, stats = step(head, batch, logp_ref)
        torch.cuda.synchronize()
        named = dict(zip(rlk.PREF_STAT_NAMES, stats.tolist()))
        print(f"step {k}: loss {loss.item():.5f}  margin {named['margin']:+.5f}  accuracy {named['accuracy']:.2f}"
              f"  ({(time.perf_counter() - t) * 1e3:.2f} ms, {batch['x'].shape[0]} tokens)")


if __name__ == "__main__":
    main()
