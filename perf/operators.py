"""The operators around the log-probability path, as cases to measure.

A preference-training step runs, between the last block's activations and the
weights' gradients:

  x -> linear (bias, activation, residual) -> norm -> LM head + scorer -> preference loss
    -> LM head backward -> norm backward -> linear backward

The LM head and the scorer are the library's; the cases here are the other
operators: the matrix product with its fused epilogue, layer / RMS norm, the
8-bit activation checkpoints that the backward passes read in place of the
activations, and the paired preference loss.

``own`` chooses who computes: False is the plain form in elementary torch
operations at 32 bits, True makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32            # elements that share one checkpoint scale
BF16, F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # serving: the final norm of one token's hidden state
        dict(name="norm_one_token", op="norm", T=1, H=4096, kind="rms", bias=False, dtype="bf16", dy="", ckpt=False),
        # training: the final norm and its backward, whose gradient comes from the LM head in fp32
        dict(name="norm_train", op="norm", T=16384, H=4096, kind="rms", bias=False, dtype="bf16", dy="f32", ckpt=False),
        # training, an odd width: rows that start on no 16-byte boundary
        dict(name="norm_train_odd", op="norm", T=4099, H=5003, kind="layer", bias=True, dtype="bf16", dy="bf16", ckpt=False),
        # training with the norm's input kept in 8 bits between forward and backward
        dict(name="norm_train_checkpoint", op="norm", T=16384, H=4096, kind="layer", bias=True, dtype="bf16", dy="bf16", ckpt=True),
        # the activations of eight long responses into their checkpoint and back
        dict(name="checkpoint_long", op="checkpoint", T=55296, H=4096, dtype="bf16"),
        # a ragged fp32 activation: the last block of each row is short
        dict(name="checkpoint_odd", op="checkpoint", T=777, H=1003, dtype="f32"),
        # serving: one token through a projection (bound by the weight's bytes)
        dict(name="linear_one_token", op="linear", M=1, N=4096, K=4096, act="silu", bias=True, residual=True, preact=False),
        # a ragged batch through a projection whose rows start on no 16-byte boundary
        dict(name="linear_odd", op="linear", M=1531, N=2050, K=1001, act="gelu", bias=True, residual=True, preact=True),
        # training: a batch of prompts and responses through an output projection
        dict(name="linear_train", op="linear", M=16384, N=4096, K=4096, act="gelu", bias=True, residual=True, preact=True),
        # training: its backward, the input read from its 8-bit checkpoint
        dict(name="linear_backward", op="linear_backward", M=8192, N=4096, K=4096, act="silu", ckpt=True),
        # the smallest preference batch: four pairs of short responses
        dict(name="preference_small", op="preference", pairs=4, lo=16, hi=256, loss="sigmoid", smoothing=0.0, mean=False, ref=True),
        # a large preference batch of long responses
        dict(name="preference_large", op="preference", pairs=2048, lo=256, hi=2048, loss="sigmoid", smoothing=0.1, mean=False, ref=True),
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
    return max(lo, max(m << a for m in (4, 5, 7) for a in range(4, 12) if m << a <= v))


def draw(rng):
    op = rng.choice(["norm", "norm", "checkpoint", "linear", "linear", "linear_backward", "preference"])
    if op == "norm":
        H = _width(rng, 64, 16384)
        T = _spread(rng, 1, max(1, min(32768, (1 << 26) // H)))
        train = rng.random() < 0.75
        return dict(op=op, T=T, H=H, kind=rng.choice(["layer", "rms"]), bias=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    dy=rng.choice(["bf16", "f32"]) if train else "", ckpt=train and rng.random() < 0.4)
    if op == "checkpoint":
        H = _width(rng, 32, 16384)
        return dict(op=op, T=_spread(rng, 1, max(1, min(55296, (1 << 27) // H))), H=H, dtype=rng.choice(["bf16", "f32"]))
    if op == "linear":
        N, K = _width(rng, 128, 16384), _width(rng, 128, 16384)
        M = _spread(rng, 1, max(1, min(16384, (1 << 38) // (N * K))))
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(["none", "gelu", "silu", "relu"]), bias=rng.random() < 0.7, residual=rng.random() < 0.6,
                    preact=rng.random() < 0.5)
    if op == "linear_backward":
        N, K = _width(rng, 128, 8192), _width(rng, 128, 8192)
        M = _spread(rng, 64, max(64, min(8192, (1 << 37) // (N * K))))
        return dict(op=op, M=M, N=N, K=K, act=rng.choice(["none", "gelu", "silu"]), ckpt=rng.random() < 0.5)
    lo = _spread(rng, 1, 512)
    hi = _spread(rng, lo, 4096)
    return dict(op=op, pairs=_spread(rng, 1, max(1, min(2048, (1 << 21) // hi))), lo=lo, hi=hi, loss=rng.choice(["sigmoid", "sigmoid", "ipo", "hinge"]),
                smoothing=rng.choice([0.0, 0.1]), mean=rng.random() < 0.3, ref=rng.random() < 0.8)


# ------------------------------------------------------------------ inputs
def _dtype(name):
    return {"bf16": BF16, "f32": F32}[name]


def _activations(T, H, dtype, g):
    """Hidden states as a trained model has them: Gaussian rows, a gain for
    each channel, a few channels an order of magnitude above the rest."""
    gain = torch.exp(0.3 * torch.randn(H, device="cuda", generator=g))
    gain[torch.randint(0, H, (max(1, H // 512),), device="cuda", generator=g)] *= 12.0
    shift = 0.1 * torch.randn(H, device="cuda", generator=g)
    return torch.randn(T, H, device="cuda", generator=g).mul_(gain).add_(shift).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)
    s = dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = _activations(T, H, _dtype(case["dtype"]), g)
        s["w"] = 1.0 + 0.1 * randn(H)
        s["b"] = 0.1 * randn(H) if case["bias"] else None
        if case["dy"]:
            s["g"] = (randn(T, H) * 1e-2).to(_dtype(case["dy"]))
    elif case["op"] == "checkpoint":
        s["x"] = _activations(case["T"], case["H"], _dtype(case["dtype"]), g)
    elif case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = randn(M, K).to(BF16)
        s["w"] = (randn(N, K) / math.sqrt(K)).to(BF16)
        s["b"] = 0.1 * randn(N) if case["bias"] else None
        s["r"] = randn(M, N).to(BF16) if case["residual"] else None
    elif case["op"] == "linear_backward":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(M, K, BF16, g)
        s["w"] = (randn(N, K) / math.sqrt(K)).to(BF16)
        s["z"] = randn(M, N).to(BF16) if case["act"] != "none" else None
        s["g"] = (randn(M, N) * 1e-2).to(BF16)
        if case["ckpt"]:   # what the forward kept: 8-bit codes and the blocks' scales
            k = _step_exponent(x.float())
            blocks = -(-K // BLOCK)
            ldq = -(-K // 16) * 16
            codes = torch.zeros(M, ldq, device="cuda", dtype=torch.int8)
            step = torch.ldexp(torch.ones_like(k, dtype=F32), k).repeat_interleave(BLOCK, 1)[:, :K]
            codes[:, :K] = torch.round(x.float() / step).to(torch.int8)
            scales = torch.zeros(M, -(-blocks // 16) * 16, device="cuda", dtype=torch.uint8)
            scales[:, :blocks] = (k + 127).to(torch.uint8)
            s["codes"], s["scales"] = codes, scales
        else:
            s["x"] = x
    else:
        rs = np.random.RandomState(seed % (1 << 31))
        lens = np.random.RandomState(case["pairs"]).randint(case["lo"], case["hi"] + 1, 2 * case["pairs"])
        rs.shuffle(lens)                                   # the same lengths in all, in another order for each seed
        off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        n = int(off[-1])
        s["off"] = torch.from_numpy(off).cuda()
        s["lp"] = -torch.empty(n, device="cuda").exponential_(1.0, generator=g)
        s["lr"] = s["lp"] + 0.05 * randn(n) if case["ref"] else None
        m = torch.rand(n, device="cuda", generator=g) < 0.85
        empty = rs.rand(2 * case["pairs"]) < 0.02      # responses that the mask leaves nothing of
        if empty.any():
            m &= torch.from_numpy(np.repeat(~empty, lens)).cuda()
        s["lp"][~m] = -math.inf                          # what a masked place may hold
        s["mask"] = m.to(torch.uint8)
    return s


# -------------------------------------------------------------- the plain forms
def _step_exponent(x):
    """k per block of 32: the least whole number >= -126 with 127 * 2^k >= max |x|."""
    T, H = x.shape
    pad = (-H) % BLOCK
    a = torch.nn.functional.pad(x.abs(), (0, pad)).view(T, -1, BLOCK).amax(2)
    m, e = torch.frexp(a)
    k = e - 7 + (m > 127.0 / 128.0).to(torch.int32)
    return torch.where(a > 0, k, torch.full_like(k, -126)).clamp_min(-126).to(torch.int32)


def _through_checkpoint(x):
    """The values that the 8-bit checkpoint of x stands for."""
    x = x.float()
    k = _step_exponent(x).repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    return torch.ldexp(torch.round(torch.ldexp(x, -k)), k)


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z.clamp_min(0.0) if act == "relu" else z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_norm(s):
    x, eps = s["x"].float(), 1e-5
    if s["kind"] == "layer":
        mean = x.mean(1)
        c = x - mean[:, None]
    else:
        mean, c = None, x
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    out = {"y": y.to(s["x"].dtype), "rstd": rstd}
    if mean is not None:
        out["mean"] = mean
    if s["dy"]:
        if s["ckpt"]:
            c = _through_checkpoint(s["x"])
            c = c - mean[:, None] if mean is not None else c
        dy, xhat = s["g"].float(), c * rstd[:, None]
        d = dy * s["w"]
        dx = d - xhat * (d * xhat).mean(1, keepdim=True)
        if mean is not None:
            dx = dx - d.mean(1, keepdim=True)
        out["dx"] = (dx * rstd[:, None]).to(s["x"].dtype)
        out["dw"] = (dy * xhat).sum(0)
        if s["b"] is not None:
            out["db"] = dy.sum(0)
    return out


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(BF16), "z": z.to(BF16)} if s["preact"] else {"y": y.to(BF16)}


def _plain_linear_backward(s):
    K = s["K"]
    if s["ckpt"]:
        k = (s["scales"].to(torch.int32) - 127).repeat_interleave(BLOCK, 1)[:, :K]
        x = torch.ldexp(s["codes"][:, :K].float(), k)
    else:
        x = s["x"].float()
    dz = s["g"].float()
    if s["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), s["act"])
    return {"dx": (dz @ s["w"].float()).to(BF16), "dw": (dz.t() @ x).to(BF16), "db": dz.sum(0)}


def _plain_preference(s):
    beta, P, n = 0.1, s["pairs"], s["lp"].numel()
    lens = (s["off"][1:] - s["off"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(2 * P, device="cuda"), lens, output_size=n)
    m = s["mask"] != 0
    d = s["lp"] - s["lr"] if s["ref"] else s["lp"]
    zero = torch.zeros(2 * P, device="cuda")
    delta = zero.index_add(0, seq, torch.where(m, d, 0.0))
    count = zero.index_add(0, seq, m.float())
    scale = 1.0 / count.clamp_min(1.0) if s["mean"] else torch.ones_like(count)
    reward = beta * delta * scale
    live = (count[0::2] > 0) & (count[1::2] > 0)
    h = reward[0::2] - reward[1::2]
    eps = s["smoothing"]
    if s["loss"] == "sigmoid":
        soft = lambda v: torch.clamp_min(-v, 0.0) + torch.log1p(torch.exp(-v.abs()))
        loss = (1.0 - eps) * soft(h) + eps * soft(-h)
        slope = -(1.0 - eps) / (1.0 + torch.exp(h)) + eps / (1.0 + torch.exp(-h))
    elif s["loss"] == "hinge":
        loss, slope = torch.clamp_min(1.0 - h, 0.0), -(h < 1.0).float()
    else:
        loss, slope = (h / beta - 0.5 / beta) ** 2, 2.0 * (h / beta - 0.5 / beta) / beta
    loss, slope = torch.where(live, loss, 0.0), torch.where(live, slope, 0.0) / P
    per_seq = torch.stack([slope, -slope], 1).reshape(-1) * beta * scale
    return {"loss": loss.sum() / P, "grad": torch.where(m, per_seq[seq], 0.0), "reward": reward}


# -------------------------------------------------------------- the library's calls
def _own(s):
    import entropy_logits_bf16_gb300 as rlk

    acts = {"none": rlk.ACT_NONE, "gelu": rlk.ACT_GELU, "silu": rlk.ACT_SILU, "relu": rlk.ACT_RELU}
    if s["op"] == "norm":
        kind = rlk.NORM_LAYER if s["kind"] == "layer" else rlk.NORM_RMS
        ck = rlk.new_checkpoint(s["T"], s["H"], s["x"].device) if s["ckpt"] else None
        y, mean, rstd = rlk.norm(s["x"], s["w"], s["b"], kind=kind, eps=1e-5, checkpoint=ck)
        out = {"y": y, "rstd": rstd}
        if mean is not None:
            out["mean"] = mean
        if s["dy"]:
            out["dx"], out["dw"], db = rlk.norm_backward(s["g"], ck if ck is not None else s["x"], s["w"], mean, rstd, kind=kind,
                                                         grad_dtype=s["x"].dtype, want_bias_grad=s["b"] is not None)
            if db is not None:
                out["db"] = db
        return out
    if s["op"] == "checkpoint":
        return rlk.checkpoint_unpack(rlk.checkpoint_pack(s["x"]), dtype=s["x"].dtype)
    if s["op"] == "linear":
        got = rlk.linear(s["x"], s["w"], s["b"], s["r"], activation=acts[s["act"]], return_preact=s["preact"])
        return {"y": got[0], "z": got[1]} if s["preact"] else {"y": got}
    if s["op"] == "linear_backward":
        x = rlk.Checkpoint(s["codes"], s["scales"], s["M"], s["K"]) if s["ckpt"] else s["x"]
        dx, dw, db = rlk.linear_backward(s["g"], x, s["w"], s["z"], activation=acts[s["act"]], weight_grad_dtype=BF16)
        return {"dx": dx, "dw": dw, "db": db}
    kinds = {"sigmoid": rlk.PREF_SIGMOID, "ipo": rlk.PREF_IPO, "hinge": rlk.PREF_HINGE}
    loss, grad, reward, _ = rlk.preference_loss(s["lp"], s["lr"], s["off"], loss_mask=s["mask"], loss_type=kinds[s["loss"]], beta=0.1,
                                                label_smoothing=s["smoothing"], length_normalise=s["mean"], want_stats=False)
    return {"loss": loss.reshape(()), "grad": grad, "reward": reward}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _plain_norm(state)
    if state["op"] == "checkpoint":
        return _through_checkpoint(state["x"]).to(state["x"].dtype)
    if state["op"] == "linear":
        return _plain_linear(state)
    if state["op"] == "linear_backward":
        return _plain_linear_backward(state)
    return _plain_preference(state)


# -------------------------------------------------------------- work and exact values
def work(case):
    size = {"bf16": 2, "f32": 4, "": 0}
    if case["op"] == "norm":
        T, H, e = case["T"], case["H"], size[case["dtype"]]
        kept = 1 + 1 / BLOCK if case["ckpt"] else 0          # the checkpoint: written once, read once
        b = T * H * (2 * e + kept) + 4 * H * (2 if case["bias"] else 1) + 4 * T * (2 if case["kind"] == "layer" else 1)
        if case["dy"]:
            b += T * H * (size[case["dy"]] + (kept or e) + e) + 4 * H * (3 if case["bias"] else 2) + 8 * T
        return {"bytes": b, "flops": T * H * (18 if case["dy"] else 7)}
    if case["op"] == "checkpoint":
        n = case["T"] * case["H"]
        return {"bytes": n * (2 * size[case["dtype"]] + 2 * (1 + 1 / BLOCK)), "flops": 5 * n}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * (M * K + N * K) + 4 * N * case["bias"] + 2 * M * N * (1 + case["residual"] + case["preact"]), "flops": 2 * M * N * K}
    if case["op"] == "linear_backward":
        M, N, K = case["M"], case["N"], case["K"]
        x = (1 + 1 / BLOCK) if case["ckpt"] else 2
        return {"bytes": 2 * M * N * (1 if case["act"] == "none" else 2) + x * M * K + 2 * N * K + 2 * M * K + 2 * N * K + 4 * N, "flops": 4 * M * N * K}
    n = case["pairs"] * (case["lo"] + case["hi"])              # the expected number of tokens
    return {"bytes": n * (4 + 1 + 4 + (4 if case["ref"] else 0)) + 16 * case["pairs"], "flops": 5 * n}


def _exact_checkpoint(x):
    """64 bits: |x| / 127 <= 2^k found by the logarithm, put right by comparison."""
    T, H = x.shape
    x = torch.nn.functional.pad(x.double(), (0, (-H) % BLOCK)).unflatten(1, (-1, BLOCK))
    top = x.abs().max(2, keepdim=True).values
    k = torch.ceil(torch.log2(top / 127.0)).clamp_min(-126.0)
    k = torch.where((k > -126) & (127.0 * torch.exp2(k - 1) >= top), k - 1, k)
    k = torch.where(127.0 * torch.exp2(k) < top, k + 1, k)
    step = torch.exp2(k)
    return (torch.round(x / step) * step).flatten(1)[:, :H]


def exact(case, seed):
    s = prepare(case, seed)
    d = lambda name: s[name].double()
    if case["op"] == "checkpoint":
        return _exact_checkpoint(s["x"])
    if case["op"] == "norm":
        x, w, H = d("x"), d("w"), case["H"]
        mu = x.sum(1, keepdim=True) / H if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
        rs = ((x - mu).square().sum(1, keepdim=True) / H + 1e-5).pow(-0.5)
        y = (x - mu) * rs * w
        out = {"y": y + d("b") if case["bias"] else y, "rstd": rs[:, 0]}
        if case["kind"] == "layer":
            out["mean"] = mu[:, 0]
        if case["dy"]:
            n = ((_exact_checkpoint(s["x"]) if case["ckpt"] else x) - mu) * rs
            gw = d("g") * w
            dx = gw * H - n * torch.einsum("th,th->t", gw, n)[:, None]
            if case["kind"] == "layer":
                dx -= gw.sum(1, keepdim=True)
            out["dx"], out["dw"] = dx * rs / H, torch.einsum("th,th->h", d("g"), n)
            if case["bias"]:
                out["db"] = d("g").sum(0)
        return out
    if case["op"] in ("linear", "linear_backward"):
        Phi = lambda v: 0.5 * torch.erfc(-v * math.sqrt(0.5))
        sig = torch.sigmoid
    if case["op"] == "linear":
        z = torch.einsum("mk,nk->mn", d("x"), d("w"))
        z = z + d("b") if case["bias"] else z
        y = {"none": lambda v: v, "relu": torch.relu, "gelu": lambda v: v * Phi(v), "silu": lambda v: v * sig(v)}[case["act"]](z)
        y = y + d("r") if case["residual"] else y
        return {"y": y, "z": z} if case["preact"] else {"y": y}
    if case["op"] == "linear_backward":
        if case["ckpt"]:
            step = torch.exp2(s["scales"].double() - 127.0)
            x = (s["codes"].double().unflatten(1, (-1, 16)) * step.repeat_interleave(2, 1)[:, :s["codes"].shape[1] // 16, None]).flatten(1)[:, :case["K"]]
        else:
            x = d("x")
        dz = d("g")
        if case["act"] != "none":
            z = d("z")
            dz = dz * (Phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi) if case["act"] == "gelu" else sig(z) * (1 + z * sig(-z)))
        return {"dx": torch.einsum("mn,nk->mk", dz, d("w")), "dw": torch.einsum("mn,mk->nk", dz, x), "db": dz.sum(0)}
    beta, P = 0.1, case["pairs"]
    off = s["off"].long()
    m = s["mask"].double()
    diff = torch.where(s["mask"] != 0, d("lp") - (d("lr") if case["ref"] else 0.0), 0.0)
    run_d, run_m = (torch.nn.functional.pad(torch.cumsum(v, 0), (1, 0)) for v in (diff, m))
    total, count = run_d[off[1:]] - run_d[off[:-1]], run_m[off[1:]] - run_m[off[:-1]]
    per = 1.0 / count.clamp_min(1.0) if case["mean"] else torch.ones_like(count)
    reward = beta * total * per
    pair = reward.view(P, 2)
    h = pair[:, 0] - pair[:, 1]
    live = (count.view(P, 2).min(1).values > 0).double()
    e = case["smoothing"]
    if case["loss"] == "sigmoid":
        lo = -(1 - e) * torch.nn.functional.logsigmoid(h) - e * torch.nn.functional.logsigmoid(-h)
        dh = -(1 - e) * torch.sigmoid(-h) + e * torch.sigmoid(h)
    elif case["loss"] == "hinge":
        lo, dh = torch.relu(1 - h), -(h < 1).double()
    else:
        lo, dh = ((h - 0.5) / beta).square(), 2 * (h - 0.5) / beta ** 2
    sign = torch.tensor([1.0, -1.0], device="cuda", dtype=torch.float64)
    grad = torch.repeat_interleave(((dh * live)[:, None] * sign).flatten() * beta * per / P, off[1:] - off[:-1]) * m
    return {"loss": (lo * live).mean(), "grad": grad, "reward": reward}
