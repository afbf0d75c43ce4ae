"""Float64 references of the mixture-of-experts operators, straight from the formulas in
``include/moe.h``, on whatever device the inputs are, and the rounding bounds of the tests."""
import math

import torch

GATED = ("swiglu", "geglu", "reglu", "glu")
ACTS = ("none", "relu", "relu_sq", "gelu_tanh") + GATED
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U32 = torch.finfo(torch.float32).eps / 2


def half_step(dtype):
    """What rounding to dtype is off by at most, relative to the value."""
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Half the distance of dtype's smallest values: what rounding near zero is off by at most."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def fn(act, z):
    """f(z), f'(z)"""
    if act in ("swiglu", "glu"):
        s = torch.sigmoid(z)
        return (z * s, s * (1 + z * (1 - s))) if act == "swiglu" else (s, s * (1 - s))
    if act in ("gelu_tanh", "geglu"):
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "none":
        return z, torch.ones_like(z)
    r = z.clamp(min=0)
    return (r * r, 2 * r) if act == "relu_sq" else (r, (z > 0).to(z.dtype))


def route(logits, k, score, renorm):
    x = logits.double()
    ids = torch.sort(x.cpu(), dim=1, descending=True, stable=True)[1][:, :k].to(x.device)
    if score == "softmax":
        top = x.max(dim=1, keepdim=True)[0]
        e = torch.where(top == -math.inf, torch.zeros_like(x), torch.exp(x - top))
        total = e.sum(dim=1, keepdim=True)
        p = e / torch.where(total == 0, torch.ones_like(total), total)
    else:
        p = torch.sigmoid(x)
    w = p.gather(1, ids)
    if renorm:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total == 0, torch.zeros_like(w), w / total)
    return ids, w, p


def route_bwd(logits, ids, dweights, score, renorm):
    """Through the Jacobian of the weights, entry by entry: dw_j / dx_e."""
    _, _, p = route(logits, 1, score, False)
    g = dweights.double()
    pc = p.gather(1, ids)
    if renorm:   # w = pc / sum(pc)
        total = pc.sum(dim=1, keepdim=True)
        safe = torch.where(total == 0, torch.ones_like(total), total)
        g = torch.where(total == 0, torch.zeros_like(g), (g - (g * pc / safe).sum(dim=1, keepdim=True)) / safe)
    dp = torch.zeros_like(p).scatter_add_(1, ids, g)
    if score == "softmax":
        return p * (dp - (dp * p).sum(dim=1, keepdim=True))
    return dp * p * (1 - p)


def sort(ids, E):
    flat = ids.reshape(-1).long().cpu()
    key = torch.where((flat < 0) | (flat >= E), torch.full_like(flat, E), flat)
    slot_of = torch.tensor(sorted(range(flat.numel()), key=lambda i: (int(key[i]), i)), dtype=torch.long)
    row_of = torch.empty_like(slot_of)
    row_of[slot_of] = torch.arange(flat.numel())
    offsets = torch.tensor([int((key < e).sum()) for e in range(E + 1)])
    return offsets, row_of, slot_of


def spans(offsets, M):
    """(expert, first row, end row) of every expert, offsets None: one with all rows."""
    if offsets is None:
        return [(None, 0, M)]
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def _w(w, e):
    return (w if e is None else w[e]).double()


def linear(act, x, w, w_up, bias, bias_up, residual, offsets):
    """y, preact, and for the bounds: the sums of absolute products behind z (and u)."""
    M, N = x.shape[0], w.shape[-2]
    gated = act in GATED
    y = torch.zeros(M, N, dtype=torch.float64, device=x.device)
    pre = torch.zeros(M, 2 * N if gated else N, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(pre)
    for e, a, b in spans(offsets, M):
        if a == b:
            continue
        xs = x[a:b].double()
        for i, (m, t) in enumerate(((w, bias), (w_up, bias_up))[: 2 if gated else 1]):
            z = xs @ _w(m, e).T
            q = xs.abs() @ _w(m, e).abs().T
            if t is not None:
                z = z + _w(t, e)
                q = q + _w(t, e).abs()
            pre[a:b, i * N:(i + 1) * N] = z
            mag[a:b, i * N:(i + 1) * N] = q
        f = fn(act, pre[a:b, :N])[0]
        y[a:b] = f * pre[a:b, N:] if gated else f
    if residual is not None:
        y = y + residual.double()
    return y, pre, mag


def linear_dz(act, dy, preact, N):
    dy = dy.double()
    if act == "none":
        return dy
    pre = preact.double()
    f, df = fn(act, pre[:, :N])
    return torch.cat([dy * pre[:, N:] * df, dy * f], dim=1) if act in GATED else dy * df


def linear_bwd(act, dy, x, w, w_up, preact, offsets):
    """dx, [dw, dw_up], [dbias, dbias_up], and the bounds' magnitudes: for each the sum of absolute
    products, the root of the sum of their squares, and the sum of the absolute factors dz meets."""
    M, N, gated = x.shape[0], w.shape[-2], act in GATED
    dz = linear_dz(act, dy, preact, N)
    zero = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=x.device)   # noqa: E731
    dx, ax, qx, fx = zero(x), zero(x), zero(x), zero(x)
    ws = [w, w_up] if gated else [w]
    dw, aw, qw, fw = ([zero(t) for t in ws] for _ in range(4))
    db = [zero(t[..., 0]) for t in ws]
    ab = [zero(t[..., 0]) for t in ws]
    for e, a, b in spans(offsets, M):
        if a == b:
            continue
        xs = x[a:b].double()
        for i, m in enumerate(ws):
            d, wm = dz[a:b, i * N:(i + 1) * N], _w(m, e)
            dx[a:b] += d @ wm
            ax[a:b] += d.abs() @ wm.abs()
            qx[a:b] += (d * d) @ (wm * wm)
            fx[a:b] += wm.abs().sum(dim=0)
            at = slice(None) if e is None else e
            dw[i][at] = d.T @ xs
            aw[i][at] = d.abs().T @ xs.abs()
            qw[i][at] = (d * d).T @ (xs * xs)
            fw[i][at] = xs.abs().sum(dim=0).expand_as(wm)
            db[i][at] = d.sum(dim=0)
            ab[i][at] = d.abs().sum(dim=0)
    return dict(dz=dz, dx=(dx, ax, qx.sqrt(), fx), dw=list(zip(dw, aw, [q.sqrt() for q in qw], fw)), db=list(zip(db, ab)))


# ---- bounds -------------------------------------------------------------------------------------

# The activations are computed in fp32 from the hardware exponential and reciprocal: each of the few
# steps is off by a few half steps relative to its result, the exponential's argument by a half step
# relative to itself (up to |z| half steps of the result, the exponential of z > 0 entering as a
# reciprocal), and 1 + tanh cancels (half a step of 1, times z / 2). 16 (1 + |z|) half steps cover f
# and f' against |z| + 1.
def act_err(z):
    return 16 * U32 * (1 + z.abs()) ** 2


# A sum of n products in fp32, whatever the order, is off by at most n half steps of the sum of the
# absolute products; MFMA may add several products before it rounds, or round each: 2 n covers both.
def sum_err(n, mag):
    return 2 * (n + 2) * U32 * mag


# |f'| of every activation on the values here (gelu and silu stay below 1.13; relu^2: 2 z)
def slope(act, z):
    return 2 * z.abs() + 1e-3 if act == "relu_sq" else torch.full_like(z, 1.13)


def linear_bound(act, dtype, K, y, pre, mag, N):
    z, mz = pre[:, :N], mag[:, :N]
    dz = sum_err(K, mz)
    f = fn(act, z)[0]
    ef = dz if act == "none" else slope(act, z.abs() + dz) * dz + act_err(z) * (1 + z.abs() if act == "relu_sq" else 1)
    if act in GATED:
        u, du = pre[:, N:], sum_err(K, mag[:, N:])
        ef = ef * (u.abs() + du) + f.abs() * du
    return (half_step(dtype) + 4 * U32) * (y.abs() + ef) + ef + floor_of(dtype)


def check(name, got, ref, bound):
    got = got.double().to(ref.device)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: values that are not finite"
    bad = (got - ref).abs() > bound
    worst = ((got - ref).abs() / bound.clamp(min=1e-300)).max().item() if ref.numel() else 0.0
    print(f"    {name:>10}: worst error {worst:.3f} of its bound", flush=True)
    if bad.any():
        at = tuple(int(i) for i in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values out of bounds, first at {at}: "
                             f"{got[at].item()!r}, not {ref[at].item()!r} +- {bound[at].item():.3e}")
