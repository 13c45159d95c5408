"""Plain 64-bit forms of the layers around the LM head, for the tests."""
import torch

EPS32 = 2.0 ** -24     # half an ulp of 1 in fp32: one rounding's relative error
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def norm64(x, w, b, rms, eps):
    """(y, mean, rstd) of layer / RMS norm in 64 bits."""
    x = x.double()
    m = torch.zeros_like(x[:, 0]) if rms else x.mean(1)
    c = x - m[:, None]
    r = (c.square().mean(1) + eps).rsqrt()
    y = c * r[:, None]
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, m, r


def norm_grad64(dy, x, w, m, r, rms):
    """(dx, dw, db) by the formula, from the statistics given."""
    dy, h = dy.double(), (x.double() - m.double()[:, None]) * r.double()[:, None]
    g = dy if w is None else dy * w.double()
    dx = g - h * (g * h).mean(1, keepdim=True)
    if not rms:
        dx = dx - g.mean(1, keepdim=True)
    return dx * r.double()[:, None], (dy * h).sum(0), dy.sum(0)


def checkpoint64(x):
    """(codes, scale bytes, values) of the 8-bit checkpoint of x, block by
    block, the step found by trying every exponent."""
    T, H = x.shape
    nb = -(-H // 32)
    x = x.double().cpu()
    codes = torch.zeros((T, H), dtype=torch.int8)
    scales = torch.zeros((T, nb), dtype=torch.uint8)
    vals = torch.zeros((T, H), dtype=torch.float64)
    ks = 2.0 ** torch.arange(-126, 123, dtype=torch.float64)   # up to the largest fp32 (k = 122)
    for b in range(nb):
        blk = x[:, 32 * b:32 * b + 32]
        amax = blk.abs().amax(1)
        i = (127.0 * ks[None, :] < amax[:, None]).sum(1).clamp_max(ks.numel() - 1)
        step = ks[i]
        bad = ~torch.isfinite(amax)
        q = torch.where(bad[:, None], 0.0, torch.round(blk / step[:, None]))   # half to even
        q = torch.where((step == 2.0 ** 122)[:, None], q.clamp(-63, 63), q)      # 64 steps of 2^122 overflow
        codes[:, 32 * b:32 * b + 32] = q.to(torch.int8)
        scales[:, b] = torch.where(bad, 255, i + 1).to(torch.uint8)
        vals[:, 32 * b:32 * b + 32] = torch.where(bad[:, None], float("nan"), q * step[:, None])
    return codes, scales, vals


def rows(T, H, dtype, seed, device="cuda", odd_layout=False):
    """Hidden states with a gain and a shift per channel and a few large
    channels; odd_layout: rows in a wider buffer, starting off 16 bytes."""
    g = torch.Generator().manual_seed(seed)
    gain = torch.exp(0.3 * torch.randn(H, generator=g))
    gain[torch.randint(0, H, (max(1, H // 512),), generator=g)] *= 12.0
    x = (torch.randn(T, H, generator=g) * gain + 0.1 * torch.randn(H, generator=g)).to(dtype).to(device)
    if not odd_layout:
        return x
    buf = torch.full((T, H + 5), float("nan"), dtype=dtype, device=device)
    buf[:, 3:3 + H] = x
    return buf[:, 3:3 + H]


def randn(shape, seed, dtype=torch.float32, scale=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(device)


def preference64(lp, ref, mask, off, kind, beta, smoothing, margin, mean):
    """(loss, grad, reward, stats) of the preference loss, pair by pair in 64
    bits; kind 0 sigmoid, 1 IPO, 2 hinge."""
    import math
    lp = lp.double().cpu()
    ref = None if ref is None else ref.double().cpu()
    P = (len(off) - 1) // 2
    grad, reward = torch.zeros_like(lp), torch.zeros(2 * P, dtype=torch.float64)
    on = [torch.arange(off[s], off[s + 1]) for s in range(2 * P)]
    if mask is not None:
        on = [i[mask.cpu()[i] != 0] for i in on]
    for s, i in enumerate(on):
        d = (lp[i] if ref is None else lp[i] - ref[i]).sum().item() if len(i) else 0.0
        reward[s] = beta * (d / len(i) if mean and len(i) else d)
    total, live = 0.0, []
    for p in range(P):
        if not len(on[2 * p]) or not len(on[2 * p + 1]):
            continue
        live.append(p)
        h = (reward[2 * p] - reward[2 * p + 1]).item() - margin
        if kind == 0:
            sp = lambda v: max(v, 0.0) + math.log1p(math.exp(-abs(v)))
            sg = lambda v: 1 / (1 + math.exp(-v)) if v > -700 else 0.0
            total += (1 - smoothing) * sp(-h) + (smoothing * sp(h) if smoothing else 0.0)
            slope = -(1 - smoothing) * sg(-h) + smoothing * sg(h)
        elif kind == 1:
            total += (h / beta - 0.5 / beta) ** 2
            slope = 2 * (h / beta - 0.5 / beta) / beta
        else:
            total += max(0.0, 1 - h)
            slope = -1.0 if h < 1 else 0.0
        for s, sign in ((2 * p, 1.0), (2 * p + 1, -1.0)):
            grad[on[s]] = sign * slope * beta / P / (len(on[s]) if mean else 1)
    rc, rr = reward[0::2][live], reward[1::2][live]
    n = max(1, len(live))
    loss = total / P if P else 0.0
    stats = torch.tensor([loss, len(live), (rc > rr).sum().item() / n, (rc - rr).sum().item() / n,
                          rc.sum().item() / n, rr.sum().item() / n], dtype=torch.float64)
    return loss, grad, reward, stats


def act64(z, act):
    """act(z) and act'(z) in 64 bits; 0 none, 1 GELU, 2 SiLU, 3 ReLU."""
    z = z.double()
    if act == 1:
        phi = 0.5 * torch.erfc(-z * 0.5 ** 0.5)
        return z * phi, phi + z * torch.exp(-0.5 * z * z) * (0.5 / torch.pi) ** 0.5
    if act == 2:
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == 3:
        return z.clamp_min(0), (z > 0).double()
    return z, torch.ones_like(z)
