"""Operators of a distillation step on the library, as cases to measure.

A teacher's top alternatives at each position are scored under the student,
whose last block is a gated feed-forward one, and the gradients of its matrices
become orthogonalised updates:

  x -> gated linear -> linear -> norm -> LM head -> log-probabilities of the teacher's tokens
    -> their backward -> ... -> gated linear backward -> orthogonalised update

The linear layer, the norm and the LM head are measured elsewhere.  The cases
here are the gated linear layer with its backward pass, the orthogonalisation,
and the log-probabilities of given tokens with the entropy and the top
alternatives, with their backward pass.

``own`` chooses who computes: False is the plain form in elementary torch
operations at 32 bits, True makes the library's calls.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
NORM_EPS = 1e-7


def listed():
    return [
        # serving: one token through a gated block's first half (bound by the two weights' bytes)
        dict(name="gated_one_token", op="gated", M=1, N=14336, K=4096, act="silu", bias=False, preact=False),
        # a ragged batch whose rows start on no 16-byte boundary, with biases
        dict(name="gated_odd", op="gated", M=1531, N=2731, K=1001, act="gelu", bias=True, preact=True),
        # training: a batch of prompts and responses, the pre-activations kept
        dict(name="gated_train", op="gated", M=8192, N=14336, K=4096, act="silu", bias=False, preact=True),
        # training: its backward (input, both weights, both biases)
        dict(name="gated_backward", op="gated_backward", M=8192, N=8192, K=4096, act="silu"),
        # the smallest update: one 256 x 256 matrix
        dict(name="orth_small", op="orth", B=1, m=256, n=256, dtype="bf16"),
        # a stack of equal matrices (heads or experts) in one call, fp32 momentum
        dict(name="orth_stack", op="orth", B=24, m=512, n=1024, dtype="f32"),
        # a tall matrix of odd sizes
        dict(name="orth_odd", op="orth", B=1, m=2731, n=1003, dtype="f32"),
        # a gated block's projection
        dict(name="orth_train", op="orth", B=1, m=4096, n=14336, dtype="bf16"),
        # serving: one sampled token's log-probability with 20 alternatives
        dict(name="tokens_one_row", op="tokens", T=1, V=151936, C=1, top=20, dtype="bf16", masked=False, train=False),
        # a rollout's log-probabilities, entropies and alternatives
        dict(name="tokens_rollout", op="tokens", T=4096, V=151936, C=1, top=20, dtype="bf16", masked=False, train=False),
        # distillation: 64 teacher tokens a position, with the entropy, forward and backward
        dict(name="tokens_distil", op="tokens", T=4096, V=151936, C=64, top=0, dtype="bf16", masked=False, train=True),
        # odd rows of fp32 logits with a constrained vocabulary (masked places hold -inf), gradients of the alternatives too
        dict(name="tokens_odd", op="tokens", T=777, V=50021, C=3, top=50, dtype="f32", masked=True, train=True),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi], odd ones among them."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v + rng.choice([0, 0, 1])))


def _width(rng, lo, hi):
    """A row width: any, or 4, 5 or 7 times a power of two, as models have it."""
    v = _spread(rng, lo, hi)
    if v < 64 or rng.random() < 0.4:
        return v
    return max(lo, max(m << a for m in (4, 5, 7) for a in range(4, 13) if m << a <= v))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "orth", "orth", "tokens", "tokens"])
    if op == "gated":
        N, K = _width(rng, 128, 16384), _width(rng, 128, 8192)
        M = _spread(rng, 1, max(1, min(8192, (1 << 38) // (N * K))))
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(["silu", "silu", "gelu", "relu", "none"]), bias=rng.random() < 0.4, preact=rng.random() < 0.5)
    if op == "gated_backward":
        N, K = _width(rng, 128, 8192), _width(rng, 128, 8192)
        M = _spread(rng, 64, max(64, min(8192, (1 << 37) // (N * K))))
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(["silu", "silu", "gelu", "relu"]))
    if op == "orth":
        m, n = _width(rng, 32, 4096), _width(rng, 32, 8192)
        if rng.random() < 0.4:
            m, n = n, m
        most = max(1, (1 << 36) // (min(m, n) ** 2 * max(m, n)))
        return dict(op=op, B=_spread(rng, 1, min(64, most)), m=m, n=n, dtype=rng.choice(["bf16", "f32"]))
    V = _spread(rng, 1000, 200000)
    T = _spread(rng, 1, max(1, min(4096, (1 << 28) // V)))
    return dict(op=op, T=T, V=V, C=_spread(rng, 1, 64), top=rng.choice([0, 1, 5, 20, 50, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                masked=rng.random() < 0.3, train=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return {"bf16": BF16, "f32": F32}[name]


def _logits(T, V, dtype, masked, g):
    """Rows as a trained model gives them: Gaussian logits with a few tokens far
    above the rest, in bf16 with many ties.  ``masked``: a tenth of the vocabulary
    is ruled out in each row by -inf."""
    out = torch.empty(T, V, dtype=dtype, device="cuda")
    for r in range(0, T, 512):
        n = min(512, T - r)
        z = torch.randn(n, V, device="cuda", generator=g).mul_(3.0)
        at = torch.randint(0, V, (n, 8), device="cuda", generator=g)
        z.scatter_add_(1, at, 2.0 + 10.0 * torch.rand(n, 8, device="cuda", generator=g))
        if masked:
            z.masked_fill_(torch.rand(n, V, device="cuda", generator=g) < 0.1, -math.inf)
        out[r:r + n] = z.to(dtype)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)
    s = dict(case)
    if case["op"] in ("gated", "gated_backward"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = randn(M, K).to(BF16)
        s["wg"], s["wu"] = (randn(N, K) / math.sqrt(K)).to(BF16), (randn(N, K) / math.sqrt(K)).to(BF16)
        if case["op"] == "gated":
            s["bg"], s["bu"] = (0.1 * randn(N), 0.1 * randn(N)) if case["bias"] else (None, None)
        else:   # what the forward kept, and the gradient that comes in
            s["gate"], s["up"] = randn(M, N).to(BF16), randn(M, N).to(BF16)
            s["dy"] = (1e-2 * randn(M, N)).to(BF16)
    elif case["op"] == "orth":
        B, m, n = case["B"], case["m"], case["n"]
        # a gradient's spectrum: a few strong directions over a noise floor
        r = max(1, min(m, n) // 8)
        x = torch.bmm(randn(B, m, r), randn(B, r, n)) / math.sqrt(r) + 0.5 * randn(B, m, n)
        s["x"] = (1e-3 * x).to(_dtype(case["dtype"]))
    else:
        T, V, C, top = case["T"], case["V"], case["C"], case["top"]
        s["z"] = _logits(T, V, _dtype(case["dtype"]), case["masked"], g)
        # the tokens asked for: half of them likely ones (the largest of a few random places), some places of a list empty
        at = torch.randint(0, V, (T, C, 16), device="cuda", generator=g)
        best = torch.gather(s["z"].float(), 1, at.view(T, -1)).view(T, C, 16).argmax(2, keepdim=True)
        pick = torch.where(torch.rand(T, C, device="cuda", generator=g) < 0.5, torch.gather(at, 2, best)[..., 0], at[..., 0])
        if C > 1:
            pick = torch.where(torch.rand(T, C, device="cuda", generator=g) < 0.05, -1, pick)
        s["ids"] = pick.to(torch.int32).contiguous()
        if case["train"]:
            s["glp"], s["gh"] = randn(T, C) / (T * C), 1e-2 * randn(T) / T
            s["gt"] = randn(T, top) / (T * top) if top else None
    return s


# -------------------------------------------------------------- the plain forms
def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z.clamp_min(0.0) if act == "relu" else z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return (z > 0).float() if act == "relu" else torch.ones_like(z)


def _plain_gated(s):
    x = s["x"].float()
    gate, up = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    if s["bias"]:
        gate, up = gate + s["bg"], up + s["bu"]
    y = (_act(gate, s["act"]) * up).to(BF16)
    return {"y": y, "gate": gate.to(BF16), "up": up.to(BF16)} if s["preact"] else {"y": y}


def _plain_gated_backward(s):
    x, dy, gate, up = s["x"].float(), s["dy"].float(), s["gate"].float(), s["up"].float()
    dg, du = dy * up * _act_slope(gate, s["act"]), dy * _act(gate, s["act"])
    dx = dg @ s["wg"].float() + du @ s["wu"].float()
    return {"dx": dx.to(BF16), "dwg": (dg.t() @ x).to(BF16), "dwu": (du.t() @ x).to(BF16), "dbg": dg.sum(0), "dbu": du.sum(0)}


def _plain_orth(s):
    a, b, c = COEFFICIENTS
    x = s["x"].float()
    if s["m"] > s["n"]:
        x = x.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NORM_EPS)
    for _ in range(5):
        p = x @ x.transpose(1, 2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.transpose(1, 2) if s["m"] > s["n"] else x).to(BF16).contiguous()


def _plain_tokens(s):
    z = s["z"].float() + 0.0
    T, V, top = s["T"], s["V"], s["top"]
    d = z - z.amax(1, keepdim=True)
    total = torch.exp(d).sum(1, keepdim=True)
    logp = d - torch.log(total)
    del d
    p = torch.exp(logp)
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    ids = s["ids"].long()
    there = ids >= 0
    lp = torch.where(there, torch.gather(logp, 1, ids.clamp_min(0)), 0.0)
    out = {"logprob": lp, "entropy": entropy}
    if top:
        order = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :top]   # equal logits: the lowest index first
        out["top_logprob"] = torch.gather(logp, 1, order)
        out["top_ids"] = torch.where(out["top_logprob"] > -math.inf, order, -1).to(torch.int32)
    if s["train"]:
        # dL/dz_i = sum of what asks for i - p_i (all of it) - g_H p_i (ln p_i + H)
        g = torch.where(there & (lp > -math.inf), s["glp"], 0.0)
        share = g.sum(1, keepdim=True)
        if top:
            gt = torch.where(out["top_ids"] >= 0, s["gt"], 0.0)
            share = share + gt.sum(1, keepdim=True)
        dz = torch.where(p > 0, -p * (share + s["gh"][:, None] * (logp + entropy[:, None])), 0.0)
        dz.scatter_add_(1, ids.clamp_min(0), g)
        if top:
            dz.scatter_add_(1, out["top_ids"].long().clamp_min(0), gt)
        out["dz"] = dz.to(s["z"].dtype)
    return out


# -------------------------------------------------------------- the library's calls
def _own(s):
    import entropy_logits_bf16_gb300 as rlk

    acts = {"none": rlk.ACT_NONE, "gelu": rlk.ACT_GELU, "silu": rlk.ACT_SILU, "relu": rlk.ACT_RELU}
    if s["op"] == "gated":
        got = rlk.gated_linear(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], activation=acts[s["act"]], return_preact=s["preact"])
        return {"y": got[0], "gate": got[1], "up": got[2]} if s["preact"] else {"y": got}
    if s["op"] == "gated_backward":
        dx, dwg, dwu, dbg, dbu = rlk.gated_linear_backward(s["dy"], s["x"], s["wg"], s["wu"], s["gate"], s["up"], activation=acts[s["act"]],
                                                           weight_grad_dtype=BF16)
        return {"dx": dx, "dwg": dwg, "dwu": dwu, "dbg": dbg, "dbu": dbu}
    if s["op"] == "orth":
        return rlk.orthogonalise(s["x"], steps=5, coefficients=COEFFICIENTS, eps=NORM_EPS)
    state = rlk.new_token_state(s["T"], s["z"].device) if s["train"] else None
    lp, entropy, top_ids, top_lp = rlk.token_logprobs(s["z"], s["ids"], 1.0, n_top=s["top"], state=state)
    out = {"logprob": lp, "entropy": entropy}
    if s["top"]:
        out["top_logprob"], out["top_ids"] = top_lp, top_ids
    if s["train"]:
        out["dz"] = rlk.token_logprobs_backward(s["z"], s["ids"], 1.0, state, s["glp"], s["gh"], top_ids=top_ids, grad_top=s["gt"])
    return out


def run(state):
    if own:
        return _own(state)
    if state["op"] == "gated":
        return _plain_gated(state)
    if state["op"] == "gated_backward":
        return _plain_gated_backward(state)
    if state["op"] == "orth":
        return _plain_orth(state)
    return _plain_tokens(state)


# -------------------------------------------------------------- work and exact values
def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "gated":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * (M * K + 2 * N * K) + 8 * N * case["bias"] + 2 * M * N * (3 if case["preact"] else 1), "flops": 4 * M * N * K}
    if case["op"] == "gated_backward":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 6 * M * N + 4 * M * K + 8 * N * K + 8 * N, "flops": 8 * M * N * K}
    if case["op"] == "orth":   # both symmetric products need one of their halves
        B, m, n = case["B"], case["m"], case["n"]
        k, l = min(m, n), max(m, n)
        return {"bytes": B * m * n * (size[case["dtype"]] + 2), "flops": 5 * B * (3 * k * k * l + k * k * k)}
    T, V, C, top = case["T"], case["V"], case["C"], case["top"]
    b = T * V * size[case["dtype"]] + T * (8 * C + 8 * top + 4)
    if case["train"]:          # the logits once more, and their gradient
        b += 2 * T * V * size[case["dtype"]] + T * (8 * C + 8 * top + 4)
    return {"bytes": b, "flops": T * V * (12 if case["train"] else 6)}


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda name: s[name].double()
    if case["op"] in ("gated", "gated_backward"):
        Phi = lambda v: 0.5 * torch.erfc(-v * math.sqrt(0.5))
        sig = torch.sigmoid
        act = {"none": lambda v: v, "relu": torch.relu, "gelu": lambda v: v * Phi(v), "silu": lambda v: v * sig(v)}[case["act"]]
    if case["op"] == "gated":
        gate, up = torch.einsum("mk,nk->mn", d("x"), d("wg")), torch.einsum("mk,nk->mn", d("x"), d("wu"))
        if case["bias"]:
            gate, up = gate + d("bg"), up + d("bu")
        y = act(gate) * up
        return {"y": y, "gate": gate, "up": up} if case["preact"] else {"y": y}
    if case["op"] == "gated_backward":
        g, u, dy = d("gate"), d("up"), d("dy")
        slope = {"none": torch.ones_like, "relu": lambda v: (v > 0).double(), "silu": lambda v: sig(v) * (1 + v * sig(-v)),
                 "gelu": lambda v: Phi(v) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)}[case["act"]](g)
        dg, du = dy * u * slope, dy * act(g)
        both = torch.cat([dg, du], 1)
        dw = torch.einsum("mn,mk->nk", both, d("x"))
        return {"dx": both @ torch.cat([d("wg"), d("wu")], 0), "dwg": dw[:case["N"]], "dwu": dw[case["N"]:], "dbg": dg.sum(0), "dbu": du.sum(0)}
    if case["op"] == "orth":
        a, b, c = COEFFICIENTS
        x = d("x")
        x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + NORM_EPS)
        eye = torch.eye(min(case["m"], case["n"]), device="cuda", dtype=torch.float64)
        for _ in range(5):
            q = torch.einsum("bij,bkj->bik", x, x) if case["m"] <= case["n"] else torch.einsum("bji,bjk->bik", x, x)
            q = a * eye + torch.bmm(q, b * eye + c * q)
            x = torch.bmm(q, x) if case["m"] <= case["n"] else torch.bmm(x, q)
        return x
    T, V, top = case["T"], case["V"], case["top"]
    keys = ("logprob", "entropy") + (("top_logprob", "top_ids") if top else ()) + (("dz",) if case["train"] else ())
    parts = {k: [] for k in keys}
    for r in range(0, T, 512):
        z = s["z"][r:r + 512].double()
        lse = torch.logsumexp(z, 1, keepdim=True)
        lp = z - lse
        p = torch.softmax(z, 1)
        h = torch.special.entr(p).sum(1)
        ids = s["ids"][r:r + 512].long()
        one = torch.nn.functional.pad(lp, (1, 0))          # place 0: an empty place of a list
        got = torch.gather(one, 1, ids + 1)
        parts["logprob"].append(got)
        parts["entropy"].append(h)
        if top:
            # unique whole keys: the logits' order (as fp32, -0 as 0), then the lower index
            bits = (s["z"][r:r + 512].float() + 0.0).view(torch.int32).long()
            key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 24) - torch.arange(V, device="cuda")
            at = torch.topk(key, top, 1, sorted=True)[1]
            tl = torch.gather(lp, 1, at)
            parts["top_logprob"].append(tl)
            parts["top_ids"].append(at.masked_fill(tl == -math.inf, -1).to(torch.int32))
        if case["train"]:
            gl, gh = d("glp")[r:r + 512], d("gh")[r:r + 512]
            gl = gl * ((ids >= 0) & (got > -math.inf))
            w = torch.zeros_like(one).scatter_add_(1, ids + 1, gl)
            if top:
                ti = parts["top_ids"][-1].long()
                w.scatter_add_(1, ti + 1, d("gt")[r:r + 512] * (ti >= 0))
            w = w[:, 1:]
            parts["dz"].append(w - p * w.sum(1, keepdim=True) - gh[:, None] * (p * h[:, None] - torch.special.entr(p)))
    return {k: torch.cat(v) for k, v in parts.items()}
