"""Plain 64-bit forms of a distillation step's operators, for the tests."""
import math

import torch

from _layers import EPS32, HALF_ULP, act64  # noqa: F401


def tokens64(z, ids, T, top):
    """(logprob, entropy, top ids, their log-probabilities, p) of the rows of z in 64 bits, row by row."""
    out = []
    for r in range(z.shape[0]):
        zr = z[r].double().cpu()
        x = zr / T
        m = x.max()
        s = torch.exp(x - m).sum()
        lp = x - m - torch.log(s)
        p = torch.exp(lp)
        h = -(p[p > 0] * lp[p > 0]).sum()
        order = sorted(range(len(zr)), key=lambda i: (-float(zr[i]), i))[:top] if top else []
        order = [i if zr[i] > -math.inf else -1 for i in order] + [-1] * (top - len(order))
        given = [0.0 if i == -1 else float(lp[i]) for i in ([] if ids is None else ids[r].reshape(-1).tolist())]
        out.append((given, float(h), order, [float(lp[i]) if i >= 0 else -math.inf for i in order], p, lp, float(x.max() + torch.log(s))))
    cols = list(zip(*out))
    t = lambda v: torch.tensor(v, dtype=torch.float64)
    return t(cols[0]), t(cols[1]), torch.tensor(cols[2], dtype=torch.int64), t(cols[3]), torch.stack(cols[4]), torch.stack(cols[5])


def tokens_grad64(z, ids, T, glp, gh, top_ids, gt):
    """(dz, the sizes of the terms it is made of) by the formula."""
    lp, h, _, _, p, logp = tokens64(z, ids, T, 0)
    R, V = p.shape
    named = torch.zeros(R, V + 1, dtype=torch.float64)
    size = torch.zeros(R, V + 1, dtype=torch.float64)

    def put(i, g):
        i, g = i.reshape(R, -1).cpu().long(), g.double().reshape(R, -1).cpu()
        out = torch.gather(torch.nn.functional.pad(logp, (0, 1), value=-math.inf), 1, torch.where(i < 0, V, i)) == -math.inf
        g = g.masked_fill(out, 0.0)
        named.scatter_add_(1, torch.where(i < 0, V, i), g)
        size.scatter_add_(1, torch.where(i < 0, V, i), g.abs())

    if glp is not None:
        put(ids, glp)
    if gt is not None:
        put(top_ids, gt)
    named, size = named[:, :V], size[:, :V]
    gh = torch.zeros(R, dtype=torch.float64) if gh is None else gh.double().cpu()
    live = torch.where(p > 0, logp, torch.zeros_like(logp))
    dz = (named - p * (named.sum(1, keepdim=True) + gh[:, None] * (live + h[:, None]))) / T
    terms = (size + p * (size.sum(1, keepdim=True) + gh.abs()[:, None] * (live.abs() + h[:, None]))) / T
    return dz, terms
