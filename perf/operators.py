"""What the mixture-of-experts operators are measured on: the router, the tokens sorted by expert
and back, the linear layer with its epilogue, and the experts' products.

    route    scores of T tokens over E experts -> the k largest, their weights, and the gradient
    tokens   rows of x in expert order, the experts' rows back to tokens with weights applied and
             a residual added, and both gradients
    linear   y = residual + act(x W^T + b), or its backward (dx, dW, db)
    experts  the same product with one weight matrix an expert, rows grouped by expert

``run`` computes each in elementary torch operations, in 32 bits, rounded once at the end; with
``own`` set it makes the calls of this package instead. ``exact`` gives the results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GATED = ("swiglu", "geglu", "reglu", "glu")


# ---- the cases --------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's router: a couple of dozen sequences, scores in fp32
        dict(name="route_decode", op="route", T=24, E=64, k=4, dtype="f32", score="softmax", renorm=True,
             back=False),
        # the router of a training batch, with its gradient
        dict(name="route_train", op="route", T=16384, E=128, k=8, dtype="bf16", score="softmax", renorm=True,
             back=True),
        # a decode step's tokens to their experts' rows and back onto the residual stream
        dict(name="tokens_decode", op="tokens", T=48, E=64, k=4, d=2048, dtype="bf16", dropped=0.0, back=False),
        # a training batch there and back, with both gradients
        dict(name="tokens_train", op="tokens", T=8192, E=64, k=6, d=2048, dtype="bf16", dropped=0.0, back=True),
        # a ragged fp32 batch that drops the assignments over its experts' capacity
        dict(name="tokens_dropped_f32", op="tokens", T=5003, E=60, k=3, d=1036, dtype="f32", dropped=0.1,
             back=True),
        # one new token through a wide projection
        dict(name="linear_one_token", op="linear", M=1, K=4096, N=11008, act="gelu_tanh", dtype="bf16", bias=True,
             residual=False, back=False),
        # a projection back onto the residual stream, prefill or training forward
        dict(name="linear_residual", op="linear", M=2048, K=4096, N=4096, act="none", dtype="bf16", bias=True,
             residual=True, back=False),
        # the backward of a feed-forward's first projection
        dict(name="linear_back", op="linear", M=8192, K=2048, N=4864, act="gelu_tanh", dtype="f16", bias=True,
             residual=False, back=True),
        # the experts' gate and up products of a decode step: most experts get a row or two, some none
        dict(name="experts_decode", op="experts", M=96, E=64, K=2048, N=1376, act="swiglu", dtype="bf16",
             bias=False, skew=0.7, dropped=0.0, back=False),
        # the same layer over a training batch, pre-activation kept
        dict(name="experts_train", op="experts", M=32768, E=32, K=2048, N=1376, act="swiglu", dtype="bf16",
             bias=True, skew=0.4, dropped=0.0, back=False),
        # and its backward
        dict(name="experts_train_back", op="experts", M=32768, E=32, K=2048, N=1376, act="swiglu", dtype="bf16",
             bias=True, skew=0.4, dropped=0.0, back=True),
        # a small fp32 model's experts, ragged, with dropped rows and experts left empty
        dict(name="experts_ragged_f32", op="experts", M=1003, E=12, K=260, N=516, act="relu_sq", dtype="f32",
             bias=True, skew=1.5, dropped=0.05, back=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi, dtype):
    q = 4 if dtype == "f32" else 8
    return max(q, _log_int(rng, lo, hi) // q * q)


def _cost(c):
    """(bytes, 16-bit matrix operations) of a case; fp32 products count sixteen times."""
    w = work(c)
    products = c["op"] in ("linear", "experts")
    return w["bytes"], w["flops"] * (16 if products and c["dtype"] == "f32" else 1)


def draw(rng):
    """One more case of the listed ones' ranges: from one token to a training batch, every type,
    either direction, widths that end inside a tile."""
    most = [max(v) for v in zip(*(_cost(c) for c in listed()))]
    while True:
        op = rng.choice(("route", "tokens", "linear", "experts"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        back = rng.random() < 0.5
        if op == "route":
            E = _log_int(rng, 4, 256)
            c = dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=rng.randint(1, min(8, E)), dtype=dtype,
                     score=rng.choice(("softmax", "sigmoid")), renorm=rng.random() < 0.5, back=back)
        elif op == "tokens":
            E = _log_int(rng, 4, 256)
            c = dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)), d=_width(rng, 64, 8192, dtype),
                     dtype=dtype, dropped=rng.choice((0.0, 0.0, 0.1)), back=back)
        else:
            act = rng.choice(("none", "none", "relu", "relu_sq", "gelu_tanh", "swiglu", "geglu", "reglu", "glu"))
            wide = 1408 if dtype == "f32" else 11008
            c = dict(op=op, M=_log_int(rng, 1, 32768), K=_width(rng, 128, wide, dtype), N=_width(rng, 128, wide, dtype),
                     act=act, dtype=dtype, bias=rng.random() < 0.6, back=back)
            if op == "linear":
                c["residual"] = not back and rng.random() < 0.5
            else:
                c.update(E=_log_int(rng, 2, 128), skew=rng.choice((0.0, 0.4, 1.0)), dropped=rng.choice((0.0, 0.05)))
        if all(a <= b for a, b in zip(_cost(c), most)):
            return c


def _counts(c):
    """Rows of each expert, most first: shares that fall off as a power of the rank."""
    kept = c["M"] - int(c["M"] * c["dropped"])
    p = np.arange(1, c["E"] + 1, dtype=np.float64) ** -c["skew"]
    n = np.floor(kept * p / p.sum()).astype(np.int64)
    left = kept - int(n.sum())
    n += left // c["E"]
    n[: left % c["E"]] += 1
    return n


def work(c):
    es = 4 if c["dtype"] == "f32" else 2
    op = c["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        byts = T * E * es + T * k * 8
        flops = T * E * 4
        if c["back"]:   # the weights' gradient in, the scores' gradient out
            byts += T * k * 4 + T * E * es
            flops += T * E * 4
        return {"bytes": byts, "flops": flops}
    if op == "tokens":
        T, E, k, d = c["T"], c["E"], c["k"], c["d"]
        n = T * k
        byts = n * 4 + (E + 1) * 4 + 2 * n * 4   # ids in, the order out
        byts += T * d * es + n * d * es          # x to the experts' rows
        byts += n * d * es + n * 4 + 2 * T * d * es   # their rows, weights and the residual to out
        flops = 2 * n * d
        if c["back"]:
            byts += T * d * es + n * d * es + n * 4   # dout in; the rows' and the weights' gradients out
            byts += n * d * es + T * d * es           # the rows' gradient in, the tokens' out
            flops += 4 * n * d
        return {"bytes": byts, "flops": flops}
    M, K, N = c["M"], c["K"], c["N"]
    g = 2 if c["act"] in GATED else 1
    if op == "experts":
        n = _counts(c)
        kept, live, mats, extra = int(n.sum()), int((n > 0).sum()), c["E"], (c["E"] + 1) * 4
    else:
        kept, live, mats, extra = M, 1, 1, 0
    flops = 2 * kept * K * N * g
    w, b = g * N * K * es, g * N * es * c["bias"]
    if not c["back"]:
        byts = M * K * es + live * (w + b) + M * N * es + extra
        byts += M * N * es * bool(c.get("residual")) + (M * N * g * es if _keeps(c) else 0)
        return {"bytes": byts, "flops": flops}
    byts = M * N * es + M * K * es + live * w + (M * N * g * es if c["act"] != "none" else 0)
    byts += M * K * es + mats * (w + b) + extra
    return {"bytes": byts, "flops": 2 * flops}


def _keeps(c):
    """Whether a forward keeps its pre-activation: a training batch does, a few tokens do not."""
    return c["act"] != "none" and c["M"] > 256


# ---- inputs -----------------------------------------------------------------------------------

def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)

    def uniform(bound, *shape):
        return torch.empty(*shape, device="cuda").uniform_(-bound, bound, generator=gen).to(dt)

    def popular(T, E):   # router scores: some experts are preferred throughout
        return normal(T, E, scale=1.5, dtype=torch.float32) + normal(1, E, scale=0.7, dtype=torch.float32)

    s = {"case": c}
    if c["op"] == "route":
        s["logits"] = popular(c["T"], c["E"]).to(dt)
        if c["back"]:
            s["dweights"] = normal(c["T"], c["k"], dtype=torch.float32)
    elif c["op"] == "tokens":
        T, E, k, d = c["T"], c["E"], c["k"], c["d"]
        score, ids = popular(T, E).topk(k, dim=1)
        ids = ids.to(torch.int32)
        if c["dropped"]:
            ids[torch.rand(T, k, device="cuda", generator=gen) < c["dropped"]] = -1
        s["ids"], s["weights"] = ids.contiguous(), torch.softmax(score, dim=1)
        s["x"], s["ys"], s["residual"] = normal(T, d), normal(T * k, d), normal(T, d)
        if c["back"]:
            s["dout"], s["dxs"] = normal(T, d), normal(T * k, d)
    else:
        M, K, N = c["M"], c["K"], c["N"]
        lead = (c["E"],) if c["op"] == "experts" else ()
        gated = c["act"] in GATED
        s["x"] = normal(M, K)
        s["w"] = uniform(K ** -0.5, *lead, N, K)
        s["w_up"] = uniform(K ** -0.5, *lead, N, K) if gated else None
        if c["op"] == "experts":
            n = torch.from_numpy(_counts(c)).cuda()[torch.randperm(c["E"], device="cuda", generator=gen)]
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        if c["back"]:
            s["dy"] = normal(M, N)
            s["preact"] = normal(M, 2 * N if gated else N, scale=0.6) if c["act"] != "none" else None
        else:
            s["bias"] = normal(*lead, N, scale=0.1) if c["bias"] else None
            s["bias_up"] = normal(*lead, N, scale=0.1) if c["bias"] and gated else None
            s["residual"] = normal(M, N) if c.get("residual") else None
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"route": _own_route, "tokens": _own_tokens, "linear": _own_linear, "experts": _own_linear}[op](s)
    if op == "route":
        return _plain_route(s)
    if op == "tokens":
        return _plain_tokens(s)
    return _plain_linear(s) if op == "linear" else _plain_experts(s)


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, : c["k"]]   # ties to the lowest expert
    if c["score"] == "softmax":
        e = torch.exp(x - x.max(dim=1, keepdim=True)[0])
        p = e / e.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    w = p.gather(1, ids)
    total = w.sum(dim=1, keepdim=True)
    if c["renorm"]:
        w = w / total
    out = {"ids": ids.to(torch.int32), "weights": w}
    if c["back"]:
        g = s["dweights"]
        if c["renorm"]:
            g = (g - (g * w).sum(dim=1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter_(1, ids, g)
        if c["score"] == "softmax":
            dx = p * (dp - (dp * p).sum(dim=1, keepdim=True))
        else:
            dx = dp * p * (1.0 - p)
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _plain_tokens(s):
    c = s["case"]
    E, k, dt = c["E"], c["k"], s["x"].dtype
    slot = s["ids"].reshape(-1).long()
    gone = (slot < 0) | (slot >= E)
    key = torch.where(gone, torch.full_like(slot, E), slot)
    slot_of = torch.sort(key, stable=True)[1]
    row_of = torch.empty_like(slot_of)
    row_of[slot_of] = torch.arange(slot_of.numel(), device=slot_of.device)
    n = (key[:, None] == torch.arange(E, device=key.device)).sum(dim=0)
    offsets = torch.cat([n.new_zeros(1), n.cumsum(0)])
    live = ~gone[slot_of]
    at = row_of.reshape(-1, k)
    w = torch.where(gone.reshape(-1, k), 0.0, s["weights"])
    xs = torch.where(live[:, None], s["x"][slot_of // k], 0.0)
    out = s["residual"].float() + (s["ys"][at].float() * w[:, :, None]).sum(dim=1)
    res = {"offsets": offsets.to(torch.int32), "row_of": row_of.to(torch.int32), "slot_of": slot_of.to(torch.int32),
           "xs": xs.to(dt), "out": out.to(dt)}
    if c["back"]:
        dout = s["dout"].float()
        dys = torch.where(live[:, None], w.reshape(-1)[slot_of][:, None] * dout[slot_of // k], 0.0)
        dw = (s["ys"][at].float() * dout[:, None, :]).sum(dim=2)
        kept = (~gone).reshape(-1, k)
        dx = (s["dxs"][at].float() * kept[:, :, None]).sum(dim=1)
        res.update(dys=dys.to(dt), dweights=torch.where(kept, dw, 0.0), dx=dx.to(dt))
    return res


def _act(name, g, u):
    if name in ("gelu_tanh", "geglu"):
        f = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    elif name == "swiglu":
        f = g / (1.0 + torch.exp(-g))
    elif name == "glu":
        f = 1.0 / (1.0 + torch.exp(-g))
    elif name == "none":
        f = g
    else:
        f = g.clamp(min=0.0)
        f = f * f if name == "relu_sq" else f
    return f * u if name in GATED else f


def _act_back(name, dy, g, u):
    """(dg, du) of the activation against dy; du is None for one that is not gated."""
    if name == "none":
        return dy, None
    if name in ("gelu_tanh", "geglu"):
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        f, df = 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)
    elif name in ("swiglu", "glu"):
        q = 1.0 / (1.0 + torch.exp(-g))
        f, df = (g * q, q * (1.0 + g * (1.0 - q))) if name == "swiglu" else (q, q * (1.0 - q))
    else:
        f, df = g.clamp(min=0.0), (g > 0.0).to(g.dtype)
        if name == "relu_sq":
            f, df = f * f, 2.0 * f
    return (dy * u * df, dy * f) if name in GATED else (dy * df, None)


def _plain_linear(s):
    c = s["case"]
    x, w, dt, gated = s["x"].float(), s["w"].float(), s["x"].dtype, c["act"] in GATED
    if not c["back"]:
        g = x @ w.t()
        u = x @ s["w_up"].float().t() if gated else None
        if c["bias"]:
            g = g + s["bias"].float()
            u = u + s["bias_up"].float() if gated else None
        y = _act(c["act"], g, u)
        if c["residual"]:
            y = y + s["residual"].float()
        out = {"y": y.to(dt)}
        if _keeps(c):
            out["preact"] = (torch.cat([g, u], dim=1) if gated else g).to(dt)
        return out
    N = c["N"]
    pre = s["preact"].float() if s["preact"] is not None else None
    dg, du = _act_back(c["act"], s["dy"].float(), pre[:, :N] if pre is not None else None, pre[:, N:] if gated else None)
    dx = dg @ w
    out = {"dw": (dg.t() @ x).to(dt)}
    if c["bias"]:
        out["dbias"] = dg.sum(dim=0).to(dt)
    if gated:
        dx = dx + du @ s["w_up"].float()
        out["dw_up"] = (du.t() @ x).to(dt)
        if c["bias"]:
            out["dbias_up"] = du.sum(dim=0).to(dt)
    out["dx"] = dx.to(dt)
    return out


def _plain_experts(s):
    """The experts that have rows as one batch of products, each padded to the longest."""
    c = s["case"]
    M, E, N, dt, gated = c["M"], c["E"], c["N"], s["x"].dtype, c["act"] in GATED
    off = s["offsets"].long()
    n = off[1:] - off[:-1]
    live = torch.nonzero(n)[:, 0]
    cap = int(n.max())
    row = off[live][:, None] + torch.arange(cap, device=off.device)
    has = torch.arange(cap, device=off.device) < n[live][:, None]
    row = torch.where(has, row, 0)

    def batch(t):   # [M, width] -> [live, cap, width], zeros past an expert's rows
        return torch.where(has[:, :, None], t.float()[row], 0.0)

    def rows(t):    # and back; rows of no expert are zero
        return t.new_zeros(M, t.shape[2]).index_put_((row[has],), t[has])

    x, w = batch(s["x"]), s["w"][live].float()
    w_up = s["w_up"][live].float() if gated else None
    if not c["back"]:
        g = torch.bmm(x, w.transpose(1, 2))
        u = torch.bmm(x, w_up.transpose(1, 2)) if gated else None
        if c["bias"]:
            g = g + s["bias"][live].float()[:, None]
            u = u + s["bias_up"][live].float()[:, None] if gated else None
        out = {"y": rows(_act(c["act"], g, u)).to(dt)}
        if _keeps(c):
            out["preact"] = rows(torch.cat([g, u], dim=2) if gated else g).to(dt)
        return out
    pre = batch(s["preact"]) if s["preact"] is not None else None
    dg, du = _act_back(c["act"], batch(s["dy"]), pre[:, :, :N] if pre is not None else None,
                       pre[:, :, N:] if gated else None)

    def each(t):    # [live, ...] -> [E, ...], zeros for an expert without rows
        return t.new_zeros(E, *t.shape[1:]).index_copy_(0, live, t).to(dt)

    dx = torch.bmm(dg, w)
    out = {"dw": each(torch.bmm(dg.transpose(1, 2), x))}
    if c["bias"]:
        out["dbias"] = each(dg.sum(dim=1))
    if gated:
        dx = dx + torch.bmm(du, w_up)
        out["dw_up"] = each(torch.bmm(du.transpose(1, 2), x))
        if c["bias"]:
            out["dbias_up"] = each(du.sum(dim=1))
    out["dx"] = rows(dx).to(dt)
    return out


# ---- this package's calls; buffers and workspaces live with the state, as a program keeps them --

def _kept(s, make):
    if "buffers" not in s:
        s["buffers"] = make()
    return s["buffers"]


def _own_route(s):
    import gated_mlp_gemms_amd as gm

    c, logits = s["case"], s["logits"]
    ids, w, dl = _kept(s, lambda: (torch.empty(c["T"], c["k"], dtype=torch.int32, device="cuda"),
                                   torch.empty(c["T"], c["k"], device="cuda"),
                                   torch.empty_like(logits) if c["back"] else None))
    gm.moe_route(logits, ids, w, score=c["score"], renorm=c["renorm"])
    out = {"ids": ids, "weights": w}
    if c["back"]:
        gm.moe_route_bwd(logits, ids, s["dweights"], dl, score=c["score"], renorm=c["renorm"])
        out["dlogits"] = dl
    return out


def _own_tokens(s):
    import gated_mlp_gemms_amd as gm

    c = s["case"]
    E, n = c["E"], c["T"] * c["k"]

    def make():
        order = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (E + 1, n, n)]
        ws = torch.empty(gm.moe_sort_workspace_bytes(n, E), dtype=torch.uint8, device="cuda")
        back = [torch.empty_like(s["ys"]), torch.empty_like(s["weights"]), torch.empty_like(s["x"])] if c["back"] else None
        return order, ws, torch.empty_like(s["ys"]), torch.empty_like(s["x"]), back

    (offsets, row_of, slot_of), ws, xs, out, back = _kept(s, make)
    gm.moe_sort(s["ids"], E, offsets, row_of, slot_of, workspace=ws)
    gm.moe_gather(s["x"], slot_of, offsets, xs)
    gm.moe_combine(s["ys"], s["weights"], row_of, offsets, out, residual=s["residual"])
    res = {"offsets": offsets, "row_of": row_of, "slot_of": slot_of, "xs": xs, "out": out}
    if c["back"]:
        dys, dw, dx = back
        gm.moe_combine_bwd(s["dout"], s["ys"], s["weights"], row_of, slot_of, offsets, dys, dw)
        gm.moe_gather_bwd(s["dxs"], row_of, offsets, dx)
        res.update(dys=dys, dweights=dw, dx=dx)
    return res


def _own_linear(s):
    import gated_mlp_gemms_amd as gm

    c, x, w, w_up = s["case"], s["x"], s["w"], s["w_up"]
    gated, keeps = c["act"] in GATED, _keeps(c)

    def make():
        desc = gm.make_linear_desc(c["M"], c["K"], c["N"], act=c["act"], dtype=x.dtype, experts=c.get("E", 0))
        ws = torch.empty(gm.linear_workspace_bytes(desc, "bwd" if c["back"] else "fwd"), dtype=torch.uint8,
                         device="cuda")
        if not c["back"]:
            out = {"y": x.new_empty(c["M"], c["N"])}
            if keeps:
                out["preact"] = x.new_empty(c["M"], 2 * c["N"] if gated else c["N"])
            return desc, ws, out
        out = {"dx": torch.empty_like(x), "dw": torch.empty_like(w)}
        if c["bias"]:
            out["dbias"] = w.new_empty(w.shape[:-1])
        if gated:
            out["dw_up"] = torch.empty_like(w)
            if c["bias"]:
                out["dbias_up"] = w.new_empty(w.shape[:-1])
        return desc, ws, out

    desc, ws, out = _kept(s, make)
    if not c["back"]:
        gm.linear_fwd(desc, x, w, out["y"], w_up=w_up, bias=s["bias"], bias_up=s["bias_up"], residual=s["residual"],
                      offsets=s.get("offsets"), preact=out.get("preact"), workspace=ws)
    else:
        gm.linear_bwd(desc, s["dy"], x, w, w_up=w_up, preact=s["preact"], offsets=s.get("offsets"), workspace=ws,
                      **out)
    return out


# ---- 64 bits ----------------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "route":
        return _exact_route(s)
    if c["op"] == "tokens":
        return _exact_tokens(s)
    return _exact_linear(s)


def _exact_route(s):
    c = s["case"]
    z = s["logits"].double().cpu().numpy()
    T, E = z.shape
    order = np.lexsort((np.broadcast_to(np.arange(E), z.shape), -z), axis=1)[:, : c["k"]]
    at = np.arange(T)[:, None]
    chosen = z[at, order]
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-z))
    soft = np.exp(z - np.logaddexp.reduce(z, axis=1, keepdims=True))
    if c["score"] == "softmax":   # renormalised over the chosen, a softmax of the chosen alone
        w = np.exp(chosen - np.logaddexp.reduce(chosen, axis=1, keepdims=True)) if c["renorm"] else soft[at, order]
    else:
        w = sig[at, order]
        w = w / w.sum(axis=1, keepdims=True) if c["renorm"] else w
    out = {"ids": torch.from_numpy(order.astype(np.int32)), "weights": torch.from_numpy(w)}
    if c["back"]:
        g = s["dweights"].double().cpu().numpy()
        mean = (g * w).sum(axis=1, keepdims=True)
        d = np.zeros_like(z)
        if c["score"] == "softmax":
            if c["renorm"]:
                d[at, order] = w * (g - mean)
            else:
                d = -soft * mean
                d[at, order] += w * g
        else:
            q = sig[at, order]
            d[at, order] = (w * (1.0 - q) * (g - mean)) if c["renorm"] else q * (1.0 - q) * g
        out["dlogits"] = torch.from_numpy(d)
    return out


def _exact_tokens(s):
    c = s["case"]
    E, k, T = c["E"], c["k"], c["T"]
    ids = s["ids"].cpu().numpy().reshape(-1)
    n = ids.size
    groups = [np.flatnonzero(ids == e) for e in range(E)]
    tail = np.flatnonzero((ids < 0) | (ids >= E))
    slot_of = np.concatenate(groups + [tail]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(g) for g in groups])])
    kept = int(offsets[-1])
    row_of = np.argsort(slot_of)
    order = torch.from_numpy(slot_of).cuda()
    live, token = order[:kept], order[:kept] // k
    w = s["weights"].double().reshape(-1)[live]
    ys = s["ys"][:kept].double()
    d = c["d"]
    xs = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    xs[:kept] = s["x"].double()[token]
    out = s["residual"].double().index_add(0, token, w[:, None] * ys)
    res = {"offsets": torch.from_numpy(offsets.astype(np.int32)), "row_of": torch.from_numpy(row_of.astype(np.int32)),
           "slot_of": torch.from_numpy(slot_of.astype(np.int32)), "xs": xs, "out": out}
    if c["back"]:
        dout = s["dout"].double()[token]
        dys = torch.zeros(n, d, dtype=torch.float64, device="cuda")
        dys[:kept] = w[:, None] * dout
        dw = torch.zeros(n, dtype=torch.float64, device="cuda")
        dw[live] = (ys * dout).sum(dim=1)
        dx = torch.zeros(T, d, dtype=torch.float64, device="cuda").index_add(0, token, s["dxs"][:kept].double())
        res.update(dys=dys, dweights=dw.reshape(T, k), dx=dx)
    return res


def _exact_gate(name, z):
    """f(z) and f'(z) of the activation's function."""
    if name in ("swiglu", "glu"):
        q = torch.sigmoid(z)
        return (z * q, q + z * q * (1.0 - q)) if name == "swiglu" else (q, q - q * q)
    if name in ("gelu_tanh", "geglu"):   # z sigmoid(2 v), v the polynomial inside the tanh
        b = 2.0 * math.sqrt(2.0 / math.pi)
        q = torch.sigmoid(b * (z + 0.044715 * z ** 3))
        return z * q, q + z * q * (1.0 - q) * b * (1.0 + 0.134145 * z ** 2)
    r = torch.relu(z)
    if name == "relu_sq":
        return r ** 2, 2.0 * r
    return (r, torch.sign(r)) if name in ("relu", "reglu") else (z, torch.ones_like(z))


def _exact_linear(s):
    c = s["case"]
    M, K, N, gated, many = c["M"], c["K"], c["N"], c["act"] in GATED, c["op"] == "experts"
    off = s["offsets"].cpu().tolist() if many else [0, M]
    ws = [s["w"], s["w_up"]] if gated else [s["w"]]
    ws = ws if many else [w[None] for w in ws]
    x = s["x"].double()

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")

    if not c["back"]:
        bs = [s["bias"], s["bias_up"]][: len(ws)] if c["bias"] else []
        bs = bs if many else [b[None] for b in bs]
        pre, y = zeros(M, N * len(ws)), zeros(M, N)
        for e in range(len(off) - 1):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            z = [x[a:b] @ w[e].double().T for w in ws]
            z = [v + t[e].double() for v, t in zip(z, bs)] if bs else z
            pre[a:b] = torch.cat(z, dim=1)
            f = _exact_gate(c["act"], z[0])[0]
            y[a:b] = f * z[1] if gated else f
        if c.get("residual"):
            y += s["residual"].double()
        return {"y": y, "preact": pre} if _keeps(c) else {"y": y}
    dy = s["dy"].double()
    dx, dw, db = zeros(M, K), [zeros(*w.shape) for w in ws], [zeros(*w.shape[:2]) for w in ws]
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        if s["preact"] is None:
            ds = [dy[a:b]]
        else:
            pre = s["preact"][a:b].double()
            f, df = _exact_gate(c["act"], pre[:, :N])
            ds = [dy[a:b] * pre[:, N:] * df, dy[a:b] * f] if gated else [dy[a:b] * df]
        for i, (d, w) in enumerate(zip(ds, ws)):
            dx[a:b] += d @ w[e].double()
            dw[i][e] = d.T @ x[a:b]
            db[i][e] = d.sum(dim=0)
    if not many:
        dw, db = [t[0] for t in dw], [t[0] for t in db]
    out = {"dw": dw[0]}
    if c["bias"]:
        out["dbias"] = db[0]
    if gated:
        out["dw_up"] = dw[1]
        if c["bias"]:
            out["dbias_up"] = db[1]
    out["dx"] = dx
    return out
