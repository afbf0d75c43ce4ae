"""Float64 references of the norm (``include/norm.h``) and of the balance loss (``include/moe.h``), straight from their
formulas, on whatever device the inputs are, with the rounding bounds of the tests."""
import math

import torch

from moe_reference import U32, half_step


def sum_of(x, residual):
    """h as it is kept: the sum rounded to x's type. (float64 holds the sum of two 16-bit or fp32 values of like size
    exactly enough that one rounding follows; the kernel's fp32 sum of 16-bit values is rounded once more at most.)"""
    return x if residual is None else (x.double() + residual.double()).to(x.dtype)


def norm_fwd(h, weight, bias, kind, eps):
    """y, mean, rstd and bounds of their errors. Every sum of d terms runs at most chain() additions deep."""
    h = h.double()
    d = h.shape[1]
    k = chain(d)
    w = weight.double() if weight is not None else torch.ones(d, dtype=torch.float64, device=h.device)
    b = bias.double() if bias is not None else torch.zeros_like(w)
    m = h.mean(dim=1) if kind == "layer" else torch.zeros(h.shape[0], dtype=torch.float64, device=h.device)
    dm = k * U32 * h.abs().mean(dim=1) if kind == "layer" else torch.zeros_like(m)
    f = h - m[:, None]
    var = (f * f).mean(dim=1)
    # of each difference u times its operands, of the sum (k + 4) u, and the mean's own error in second order
    rel_var = ((k + 6) * U32 * var + dm ** 2 + 2 * U32 * (f.abs() * (h.abs() + m.abs()[:, None])).mean(dim=1) * (kind == "layer")) / (var + eps)
    s = 1 / torch.sqrt(var + eps)
    rel_s = rel_var / 2 + 4 * U32
    y = f * s[:, None] * w + b
    df = dm[:, None] + U32 * (h.abs() + m.abs()[:, None])
    dy = (df * s[:, None] + f.abs() * s[:, None] * (rel_s + 4 * U32)[:, None]) * w.abs() + U32 * y.abs()
    return y, m, s, dy, dm, rel_s * s


def chain(d):
    """Additions one after another in a row's sum: 64 terms a thread at most, or the 16-byte pieces of a long row over 1024
    threads, then the lanes and the waves."""
    return 64 + d // 1024 + 32


def norm_bwd(dy, h, mean, rstd, weight, dresidual, kind):
    """dx, dweight, dbias and bounds."""
    dy, h, s = dy.double(), h.double(), rstd.double()[:, None]
    M, d = h.shape
    m = mean.double()[:, None] if kind == "layer" else torch.zeros_like(s)
    w = weight.double() if weight is not None else torch.ones(d, dtype=torch.float64, device=h.device)
    n = (h - m) * s
    dn = 2 * U32 * (h.abs() + m.abs()) * s
    g = dy * w
    k = chain(d)
    c1 = g.mean(dim=1, keepdim=True) * (kind == "layer")
    c2 = (g * n).mean(dim=1, keepdim=True)
    dc1 = k * U32 * g.abs().mean(dim=1, keepdim=True) * (kind == "layer")
    dc2 = ((k + 2) * U32 * (g * n).abs() + g.abs() * dn).mean(dim=1, keepdim=True)
    dx = s * (g - c1 - n * c2)
    ex = s * (dc1 + n.abs() * dc2 + dn * c2.abs() + 6 * U32 * (g.abs() + c1.abs() + (n * c2).abs()))
    if dresidual is not None:
        dx = dx + dresidual.double()
        ex = ex + U32 * dx.abs()
    # rows one after another: a thread's share of them over 512 workgroups (64 for long rows), the workgroup's 16 groups, the parts' runs
    rows = M // 64 + 100
    dw, db = (dy * n).sum(dim=0), dy.sum(dim=0)
    ew = (rows + 2) * U32 * (dy * n).abs().sum(dim=0) + (dy.abs() * dn).sum(dim=0)
    eb = rows * U32 * dy.abs().sum(dim=0)
    return dx, dw, db, ex, ew, eb


def probs(logits, score):
    """p over all experts, 0 in a token without any, and the factor that a score's own sigmoid leaves in a gradient."""
    z = logits.double()
    if score == "softmax":
        top = z.max(dim=1, keepdim=True)[0]
        e = torch.where(top == -math.inf, 0.0, torch.exp(z - top))
        rest = torch.ones_like(z)
    else:
        e = torch.where(z.max(dim=1, keepdim=True)[0] < -104, 0.0, torch.sigmoid(z))
        rest = torch.sigmoid(-z)
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total), rest


def balance(logits, ids, mask, score):
    T, E = logits.shape
    k = ids.shape[1]
    live = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask
    p, _ = probs(logits[live], score)
    n = int(live.sum())
    one = torch.nn.functional.one_hot(torch.where((ids < 0) | (ids >= E), E, ids).long()[live], E + 1)
    counts = one.sum(dim=(0, 1))[:E] if n else torch.zeros(E, dtype=torch.int64, device=logits.device)
    shares = p.sum(dim=0) / max(n, 1)
    loss = E * (counts.double() / max(n * k, 1) * shares).sum()
    return torch.cat([counts, counts.new_tensor([n])]), shares, loss


def balance_bwd(logits, counts, k, mask, dloss, score):
    """Through the Jacobian of p."""
    T, E = logits.shape
    n = int(counts[E])
    live = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask
    a = dloss * E * counts[:E].double() / max(n * n * k, 1)
    p, rest = probs(torch.where(live[:, None], logits, 0.0), score)
    d = p * rest * (a - (p * a).sum(dim=1, keepdim=True))
    size = p * rest * (a + (p * a).sum(dim=1, keepdim=True))
    return torch.where(live[:, None], d, 0.0), torch.where(live[:, None], size, 0.0)


__all__ = ["U32", "half_step", "sum_of", "norm_fwd", "norm_bwd", "chain", "probs", "balance", "balance_bwd"]
