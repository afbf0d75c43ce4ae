"""What a pre-norm layer's further operators are measured on: the norm in front of the layer, the
router's balance loss, and products in microscaled 4-bit floating point.

    norm      y = norm(x + residual) by layer norm or RMS norm, or its backward (dx, dweight, dbias)
    balance   tokens an expert, the balance loss over them, and the router's whole gradient
    quantize  rows to 4-bit blocks of 32 with a power-of-two scale each, and back to values
    mx4       y = act(x W^T + b) on 4-bit blocks, x quantised in the pass; or the backward's two
              products, dy and x quantised in the pass
    experts   the same product with one weight matrix an expert, rows grouped by expert

``run`` computes each in elementary torch operations, in 32 bits, rounded once; with ``own`` set it
makes the calls of this package instead. ``exact`` gives the results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GATED = ("swiglu", "geglu", "reglu", "glu")
EPS = 1e-5


# ---- the cases --------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's norm of the residual stream, the layer before added on the way
        dict(name="norm_decode", op="norm", M=24, d=4096, dtype="bf16", wdtype="bf16", kind="rms", bias=False,
             residual=True, back=False),
        # a training batch's layer norm, its sum with the residual kept
        dict(name="norm_train", op="norm", M=8192, d=4096, dtype="bf16", wdtype="bf16", kind="layer", bias=True,
             residual=True, back=False),
        # its backward, the residual stream's gradient added
        dict(name="norm_train_back", op="norm", M=8192, d=4096, dtype="bf16", wdtype="f32", kind="layer", bias=True,
             residual=True, back=True),
        # a small fp32 model's backward at a ragged size
        dict(name="norm_ragged_f32", op="norm", M=5003, d=1036, dtype="f32", wdtype="f32", kind="layer", bias=True,
             residual=False, back=True),
        # the balance loss of a small micro-batch, forward only (a step that logs it)
        dict(name="balance_small", op="balance", T=1000, E=60, k=4, dtype="f32", score="softmax", masked=0.0,
             back=False),
        # a training batch with padded positions: loss, and the router's gradient with the loss's in it
        dict(name="balance_train", op="balance", T=16384, E=128, k=8, dtype="bf16", score="softmax", masked=0.1,
             back=True),
        # a training batch's activations to 4 bits and back
        dict(name="quantize_rows", op="quantize", rows=8192, cols=4096, dtype="bf16", both=False),
        # a decode step's wide projection with 4-bit weights
        dict(name="mx4_decode", op="mx4", M=16, K=4096, N=11008, act="none", dtype="bf16", bias=False, back=False),
        # the same projection over a prefill or a training forward
        dict(name="mx4_prefill", op="mx4", M=4096, K=4096, N=11008, act="none", dtype="bf16", bias=True, back=False),
        # the two products of a 4-bit training backward
        dict(name="mx4_back", op="mx4", M=8192, K=2048, N=4864, act="none", dtype="bf16", bias=False, back=True),
        # a decode step's gate and up products of 4-bit experts: most get a row or two, some none
        dict(name="experts_decode", op="experts", M=96, E=64, K=2048, N=1376, act="swiglu", dtype="bf16", bias=False,
             skew=0.7, dropped=0.0),
        # the same layer over a prefill, rows dropped over the experts' capacity
        dict(name="experts_prefill", op="experts", M=32768, E=32, K=2048, N=1376, act="swiglu", dtype="bf16",
             bias=True, skew=0.4, dropped=0.05),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi, q):
    return max(q, _log_int(rng, lo, hi) // q * q)


def _cost(c):
    w = work(c)
    return w["bytes"], w["flops"]


def draw(rng):
    """One more case of the listed ones' ranges: from one token to a training batch, every type,
    either direction, widths that end inside a tile."""
    most = [max(v) for v in zip(*(_cost(c) for c in listed()))]
    while True:
        op = rng.choice(("norm", "norm", "balance", "quantize", "mx4", "experts"))
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        back = rng.random() < 0.5
        if op == "norm":
            c = dict(op=op, M=_log_int(rng, 1, 32768), d=_width(rng, 64, 16384, 4 if dtype == "f32" else 8), dtype=dtype,
                     wdtype=rng.choice((dtype, "f32")), kind=rng.choice(("layer", "rms")), residual=rng.random() < 0.5,
                     back=back)
            c["bias"] = c["kind"] == "layer" and rng.random() < 0.7
        elif op == "balance":
            E = _log_int(rng, 4, 256)
            c = dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=rng.randint(1, min(8, E)), dtype=dtype,
                     score=rng.choice(("softmax", "sigmoid")), masked=rng.choice((0.0, 0.0, 0.1, 0.5)), back=back)
        elif op == "quantize":
            c = dict(op=op, rows=_log_int(rng, 1, 16384), cols=_width(rng, 64, 11008, 32), dtype=dtype, both=back)
        else:
            act = rng.choice(("none", "none", "relu", "relu_sq", "gelu_tanh", "swiglu", "geglu", "reglu", "glu"))
            c = dict(op=op, M=_log_int(rng, 1, 32768), K=_width(rng, 128, 11008, 32), N=_width(rng, 128, 11008, 8),
                     act=act, dtype=dtype, bias=rng.random() < 0.6)
            if op == "mx4":
                c["back"] = back
                if back:
                    c.update(act="none", bias=False, N=max(32, c["N"] // 32 * 32))
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
    if op == "norm":
        M, d, ws = c["M"], c["d"], 4 if c["wdtype"] == "f32" else 2
        stats = M * (8 if c["kind"] == "layer" else 4)
        if not c["back"]:
            return {"bytes": M * d * es * (4 if c["residual"] else 2) + d * ws * (1 + c["bias"]) + stats, "flops": 8 * M * d}
        return {"bytes": M * d * es * (4 if c["residual"] else 3) + d * ws * (2 + c["bias"]) + stats, "flops": 16 * M * d}
    if op == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        byts, flops = T * E * es + T * k * 4 + (T if c["masked"] else 0) + E * 8, T * E * 5
        if c["back"]:
            byts += 2 * T * E * es + T * k * 8 + (T if c["masked"] else 0)
            flops += T * E * 10
        return {"bytes": byts, "flops": flops}
    if op == "quantize":
        n = c["rows"] * c["cols"]
        times = 2 if c["both"] else 1   # codes and scales written, read again; their values written
        return {"bytes": n * es + times * (2 * n * 17 // 32 + n * es), "flops": 4 * n * times}
    M, K, N = c["M"], c["K"], c["N"]
    g = 2 if c["act"] in GATED else 1
    if c.get("back"):
        return {"bytes": M * N * es + M * K * es + N * K * 17 // 32 + M * K * es + N * K * es, "flops": 4 * M * K * N}
    kept, live, extra = M, 1, 0
    if op == "experts":
        n = _counts(c)
        kept, live, extra = int(n.sum()), int((n > 0).sum()), (c["E"] + 1) * 4
    byts = M * K * es + live * g * (N * K * 17 // 32 + N * es * c["bias"]) + M * N * es + extra
    return {"bytes": byts, "flops": 2 * kept * K * N * g}


# ---- 4-bit blocks -----------------------------------------------------------------------------
# 32 values share the scale 2^(floor(log2 of the largest magnitude) - 2), stored as its exponent + 127 in a
# byte; a value's code is the nearest of 0 .5 1 1.5 2 3 4 6 times the scale (ties to the even code), its sign in bit 3,
# two codes a byte, the first in the low half. The scale of block b of row r is byte [b // 8, r, b % 8].

def _scale_shape(rows, K):
    return (K + 255) // 256, (rows // 4 + 1) * 4, 8


def _encode(x):
    """Codes [..., K] (0 .. 15) and scale exponents + 127 [..., K / 32] of x [..., K]."""
    b = x.float().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(dim=-1)
    e = (top.view(torch.int32) >> 23) - 2            # the exponent field; subnormal tops have 0
    e = e.clamp(min=0)
    v = b.abs() * ((254 - e) << 23).view(torch.float32)[..., None]   # times 2^(127 - e), exact
    code = ((v > 0.25).int() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    return (code + torch.where(torch.signbit(b), 8, 0)).reshape(x.shape).to(torch.uint8), e.to(torch.uint8)


def _decode(code, e):
    """The fp32 values [..., K] of codes and scale exponents + 127."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    grid = torch.cat([grid, -grid])
    v = grid[code.long()].reshape(*code.shape[:-1], -1, 32)
    unit = torch.where(e == 0, 1 << 22, e.int() << 23).view(torch.float32)   # 2^(e - 127); 2^-127 is subnormal
    return (v * unit[..., None]).reshape(code.shape)


def _pack(code, e):
    """The two tensors that hold [..., rows, K] codes and their scales."""
    rows, K = code.shape[-2:]
    S, R, _ = _scale_shape(rows, K)
    wide = torch.zeros(*code.shape[:-2], R, S * 8, dtype=torch.uint8, device=code.device)
    wide[..., :rows, : K // 32] = e
    scales = wide.reshape(*code.shape[:-2], R, S, 8).transpose(-3, -2).contiguous()
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), scales


def _unpack(codes, scales):
    rows, K = codes.shape[-2], codes.shape[-1] * 2
    code = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*codes.shape[:-1], K)
    e = scales.transpose(-3, -2).reshape(*scales.shape[:-3], scales.shape[-2], -1)[..., :rows, : K // 32]
    return code, e


def _rounded(x):
    """fp32 values of x's 4-bit blocks along its last dimension."""
    return _decode(*_encode(x))


def _rounded_t(x):
    """The same of x^T, its blocks along x's rows, which count as 0 behind the last."""
    pad = -x.shape[0] % 32
    t = torch.cat([x, x.new_zeros(pad, x.shape[1])]) if pad else x
    return _rounded(t.t().contiguous())


# ---- inputs -----------------------------------------------------------------------------------

def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)

    def weights(*shape):   # a projection's weights as a serving program keeps them
        w = torch.empty(*shape, device="cuda").uniform_(-shape[-1] ** -0.5, shape[-1] ** -0.5, generator=gen)
        return _pack(*_encode(w))

    s = {"case": c}
    op = c["op"]
    if op == "norm":
        M, d, wt = c["M"], c["d"], DTYPES[c["wdtype"]]
        channel = torch.exp(0.5 * torch.randn(d, device="cuda", generator=gen))   # a stream's channels differ in size
        x = (torch.randn(M, d, device="cuda", generator=gen) * channel + 0.3).to(dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(d, device="cuda", generator=gen)).to(wt)
        s["bias"] = normal(d, scale=0.1, dtype=wt) if c["bias"] else None
        if not c["back"]:
            s["x"], s["residual"] = x, normal(M, d) if c["residual"] else None
        else:   # what the forward kept
            s["h"], s["dy"] = x, normal(M, d)
            s["dresidual"] = normal(M, d) if c["residual"] else None
            h = x.double()
            mean = h.mean(dim=1) if c["kind"] == "layer" else torch.zeros(M, dtype=torch.float64, device="cuda")
            s["rstd"] = torch.rsqrt((h - mean[:, None]).square().mean(dim=1) + EPS).float()
            s["mean"] = mean.float() if c["kind"] == "layer" else None
    elif op == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        z = normal(T, E, scale=1.5, dtype=torch.float32) + normal(1, E, scale=0.7, dtype=torch.float32)
        s["logits"] = z.to(dt)
        s["ids"] = s["logits"].float().topk(k, dim=1)[1].to(torch.int32).contiguous()
        s["mask"] = torch.rand(T, device="cuda", generator=gen) >= c["masked"] if c["masked"] else None
        if c["back"]:
            s["dweights"] = normal(T, k, dtype=torch.float32, scale=1.0 / T)
            s["dloss"] = torch.full((1,), 0.02, device="cuda")
    elif op == "quantize":
        s["x"] = normal(c["rows"], c["cols"])
    else:
        M, K, N = c["M"], c["K"], c["N"]
        s["x"] = normal(M, K)
        if c.get("back"):
            s["dy"] = normal(M, N)
            s["w"], s["w_scales"] = weights(K, N)   # W^T, blocks along N
            return s
        lead = (c["E"],) if op == "experts" else ()
        gated = c["act"] in GATED
        s["w"], s["w_scales"] = weights(*lead, N, K)
        s["w_up"], s["w_up_scales"] = weights(*lead, N, K) if gated else (None, None)
        s["bias"] = normal(*lead, N, scale=0.1) if c["bias"] else None
        s["bias_up"] = normal(*lead, N, scale=0.1) if c["bias"] and gated else None
        if op == "experts":
            n = torch.from_numpy(_counts(c)).cuda()[torch.randperm(c["E"], device="cuda", generator=gen)]
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_norm, "balance": _own_balance, "quantize": _own_quantize, "mx4": _own_mx4,
                "experts": _own_mx4}[op](s)
    return {"norm": _plain_norm, "balance": _plain_balance, "quantize": _plain_quantize, "mx4": _plain_mx4,
            "experts": _plain_experts}[op](s)


def _plain_norm(s):
    c = s["case"]
    w, layer = s["weight"].float(), c["kind"] == "layer"
    if not c["back"]:
        out = {}
        h, dt = s["x"], s["x"].dtype
        if c["residual"]:
            h = (h.float() + s["residual"].float()).to(dt)
            out["h"] = h
        f = h.float()
        mean = f.mean(dim=1) if layer else torch.zeros(c["M"], device=f.device)
        f = f - mean[:, None]
        rstd = 1.0 / torch.sqrt((f * f).mean(dim=1) + EPS)
        y = f * rstd[:, None] * w
        if c["bias"]:
            y = y + s["bias"].float()
        out.update(y=y.to(dt), rstd=rstd)
        if layer:
            out["mean"] = mean
        return out
    dy, f, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    n = (f - s["mean"][:, None]) * r if layer else f * r
    g = dy * w
    dx = g - n * (g * n).mean(dim=1, keepdim=True)
    if layer:
        dx = dx - g.mean(dim=1, keepdim=True)
    dx = dx * r
    if c["residual"]:
        dx = dx + s["dresidual"].float()
    out = {"dx": dx.to(s["dy"].dtype), "dweight": (dy * n).sum(dim=0).to(s["weight"].dtype)}
    if c["bias"]:
        out["dbias"] = dy.sum(dim=0).to(s["weight"].dtype)
    return out


def _plain_balance(s):
    c, z = s["case"], s["logits"].float()
    T, E, k = c["T"], c["E"], c["k"]
    live = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=z.device)
    if c["score"] == "softmax":
        e = torch.exp(z - z.max(dim=1, keepdim=True)[0])
        rest = None
    else:
        e = 1.0 / (1.0 + torch.exp(-z))
        rest = 1.0 / (1.0 + torch.exp(z))
    p = torch.where(live[:, None], e / e.sum(dim=1, keepdim=True), 0.0)
    n = live.sum()
    at = torch.where(live[:, None], s["ids"].long(), E).reshape(-1)
    count = torch.zeros(E + 1, dtype=torch.int64, device=z.device).index_add_(0, at, torch.ones_like(at))
    counts = torch.cat([count[:E], n[None]])
    share = p.sum(dim=0) / n.clamp(min=1)
    f = count[:E].float() / (n.clamp(min=1) * k)
    out = {"counts": counts.to(torch.int32), "shares": share, "loss": (E * (f * share).sum()).reshape(1)}
    if c["back"]:
        a = s["dloss"] * E * f / n.clamp(min=1)
        d = p * (a - (p * a).sum(dim=1, keepdim=True))
        if rest is not None:
            d = d * rest
        # the chosen experts' weights, divided by their sum
        ids, g = s["ids"].long(), s["dweights"]
        w = e.gather(1, ids)
        w = w / w.sum(dim=1, keepdim=True)
        g = w * (g - (g * w).sum(dim=1, keepdim=True))
        if rest is not None:
            g = g * rest.gather(1, ids)
        out["dlogits"] = d.scatter_add(1, ids, g).to(s["logits"].dtype)
    return out


def _plain_quantize(s):
    c, x = s["case"], s["x"]
    out = {"values": _rounded(x).to(x.dtype)}
    if c["both"]:
        out["values_t"] = _rounded_t(x).to(x.dtype)
    return out


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


def _plain_mx4(s):
    c, dt = s["case"], s["x"].dtype
    w = _decode(*_unpack(s["w"], s["w_scales"]))
    if c["back"]:
        dx = _rounded(s["dy"]) @ w.t()
        dw = _rounded_t(s["dy"]) @ _rounded_t(s["x"]).t()
        return {"dx": dx.to(dt), "dw": dw.to(dt)}
    x = _rounded(s["x"])
    g, u = x @ w.t(), None
    if s["w_up"] is not None:
        u = x @ _decode(*_unpack(s["w_up"], s["w_up_scales"])).t()
    if c["bias"]:
        g = g + s["bias"].float()
        u = u + s["bias_up"].float() if u is not None else None
    return {"y": _act(c["act"], g, u).to(dt)}


def _plain_experts(s):
    """The experts that have rows as one batch of products, each padded to the longest."""
    c, dt = s["case"], s["x"].dtype
    M, off = c["M"], s["offsets"].long()
    n = off[1:] - off[:-1]
    live = torch.nonzero(n)[:, 0]
    cap = int(n.max())
    row = off[live][:, None] + torch.arange(cap, device=off.device)
    has = torch.arange(cap, device=off.device) < n[live][:, None]
    x = torch.where(has[:, :, None], _rounded(s["x"])[torch.where(has, row, 0)], 0.0)
    g = torch.bmm(x, _decode(*_unpack(s["w"][live], s["w_scales"][live])).transpose(1, 2))
    u = None
    if s["w_up"] is not None:
        u = torch.bmm(x, _decode(*_unpack(s["w_up"][live], s["w_up_scales"][live])).transpose(1, 2))
    if c["bias"]:
        g = g + s["bias"][live].float()[:, None]
        u = u + s["bias_up"][live].float()[:, None] if u is not None else None
    y = _act(c["act"], g, u)
    return {"y": y.new_zeros(M, c["N"]).index_put_((row[has],), y[has]).to(dt)}


# ---- this package's calls; buffers and workspaces live with the state, as a program keeps them --

def _kept(s, make):
    if "buffers" not in s:
        s["buffers"] = make()
    return s["buffers"]


def _own_norm(s):
    import gated_mlp_gemms_amd as gm

    c = s["case"]
    M, d, layer = c["M"], c["d"], c["kind"] == "layer"
    if not c["back"]:
        def make():
            out = {"y": torch.empty_like(s["x"]), "rstd": torch.empty(M, device="cuda")}
            if layer:
                out["mean"] = torch.empty(M, device="cuda")
            if c["residual"]:
                out["h"] = torch.empty_like(s["x"])
            return out

        out = _kept(s, make)
        gm.norm_fwd(s["x"], out["y"], weight=s["weight"], bias=s["bias"], residual=s["residual"], h=out.get("h"),
                    mean=out.get("mean"), rstd=out["rstd"], kind=c["kind"], eps=EPS)
        return out

    def make():
        out = {"dx": torch.empty_like(s["dy"]), "dweight": torch.empty_like(s["weight"])}
        if c["bias"]:
            out["dbias"] = torch.empty_like(s["weight"])
        return out, torch.empty(gm.norm_workspace_bytes(M, d), dtype=torch.uint8, device="cuda")

    out, ws = _kept(s, make)
    gm.norm_bwd(s["dy"], s["h"], s["rstd"], out["dx"], mean=s["mean"], weight=s["weight"], dresidual=s["dresidual"],
                dweight=out["dweight"], dbias=out.get("dbias"), kind=c["kind"], workspace=ws)
    return out


def _own_balance(s):
    import gated_mlp_gemms_amd as gm

    c, logits = s["case"], s["logits"]
    T, E = c["T"], c["E"]

    def make():
        out = {"counts": torch.empty(E + 1, dtype=torch.int32, device="cuda"), "shares": torch.empty(E, device="cuda"),
               "loss": torch.empty(1, device="cuda")}
        if c["back"]:
            out["dlogits"] = torch.empty_like(logits)
        return out, torch.empty(gm.moe_balance_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")

    out, ws = _kept(s, make)
    gm.moe_balance(logits, s["ids"], out["counts"], out["shares"], out["loss"], mask=s["mask"], score=c["score"],
                   workspace=ws)
    if c["back"]:
        gm.moe_balance_bwd(logits, s["ids"], out["counts"], out["dlogits"], mask=s["mask"], dloss=s["dloss"],
                           dweights=s["dweights"], score=c["score"], renorm=True)
    return out


def _blocks(gm, rows, K):
    return [torch.empty(shape, dtype=torch.uint8, device="cuda") for shape in gm.mx4_shapes(rows, K)]


def _own_quantize(s):
    import gated_mlp_gemms_amd as gm

    c, x = s["case"], s["x"]
    rows, cols = c["rows"], c["cols"]
    deep = (rows + 31) // 32 * 32

    def make():
        out = {"values": torch.empty_like(x)}
        if c["both"]:
            out["values_t"] = x.new_empty(cols, deep)
        return out, _blocks(gm, rows, cols), _blocks(gm, cols, deep) if c["both"] else (None, None)

    out, (codes, scales), (codes_t, scales_t) = _kept(s, make)
    gm.mx4_quantize(x, codes, scales, codes_t=codes_t, scales_t=scales_t)
    gm.mx4_dequantize(codes, scales, out["values"])
    if c["both"]:
        gm.mx4_dequantize(codes_t, scales_t, out["values_t"])
    return out


def _own_mx4(s):
    import gated_mlp_gemms_amd as gm

    c, x = s["case"], s["x"]
    M, K, N = c["M"], c["K"], c["N"]
    if not c.get("back"):
        def make():
            desc = gm.make_linear_desc(M, K, N, act=c["act"], dtype=x.dtype, experts=c.get("E", 0))
            ws = torch.empty(gm.mx4_linear_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
            return desc, ws, _blocks(gm, M, K), x.new_empty(M, N)

        desc, ws, (codes, scales), y = _kept(s, make)
        gm.mx4_quantize(x, codes, scales)
        gm.mx4_linear_fwd(desc, codes, scales, s["w"], s["w_scales"], y, w_up=s["w_up"], w_up_scales=s["w_up_scales"],
                          bias=s["bias"], bias_up=s["bias_up"], offsets=s.get("offsets"), workspace=ws)
        return {"y": y}

    def make():
        deep = (M + 31) // 32 * 32
        dx_desc = gm.make_linear_desc(M, N, K, dtype=x.dtype)       # dx [M, K] = dy [M, N] (W^T [K, N])^T
        dw_desc = gm.make_linear_desc(N, deep, K, dtype=x.dtype)    # dw [N, K] = dy^T [N, M] (x^T [K, M])^T
        need = max(gm.mx4_linear_workspace_bytes(dx_desc), gm.mx4_linear_workspace_bytes(dw_desc))
        out = {"dx": x.new_empty(M, K), "dw": x.new_empty(N, K)}
        return (dx_desc, dw_desc, torch.empty(need, dtype=torch.uint8, device="cuda"), _blocks(gm, M, N),
                _blocks(gm, N, deep), _blocks(gm, K, deep), out)

    dx_desc, dw_desc, ws, (g, gs), (gt, gts), (xt, xts), out = _kept(s, make)
    gm.mx4_quantize(s["dy"], g, gs, codes_t=gt, scales_t=gts)
    gm.mx4_quantize(x, codes_t=xt, scales_t=xts)
    gm.mx4_linear_fwd(dx_desc, g, gs, s["w"], s["w_scales"], out["dx"], workspace=ws)
    gm.mx4_linear_fwd(dw_desc, gt, gts, xt, xts, out["dw"], workspace=ws)
    return out


# ---- 64 bits ----------------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "balance": _exact_balance, "quantize": _exact_quantize, "mx4": _exact_mx4,
            "experts": _exact_mx4}[c["op"]](s)


def _exact_norm(s):
    c = s["case"]
    w, layer = s["weight"].double(), c["kind"] == "layer"
    if not c["back"]:
        out = {}
        h = s["x"].double()
        if c["residual"]:
            h = h + s["residual"].double()
            out["h"] = h
            h = h.to(s["x"].dtype).double()   # the norm is of the stream as it is kept
        var, mean = torch.var_mean(h, dim=1, correction=0)
        if not layer:
            var, mean = torch.linalg.vector_norm(h, dim=1) ** 2 / c["d"], torch.zeros_like(mean)
        rstd = (var + EPS) ** -0.5
        out["y"] = torch.addcmul(s["bias"].double() if c["bias"] else w.new_zeros(()), (h - mean[:, None]) * rstd[:, None], w)
        out["rstd"] = rstd
        if layer:
            out["mean"] = mean
        return out
    r = s["rstd"].double()
    n = s["h"].double()
    n = (n - s["mean"].double()[:, None] if layer else n) * r[:, None]
    dy = s["dy"].double()
    g = dy * w
    d = c["d"]
    along = torch.einsum("md,md->m", g, n) / d
    dx = g - along[:, None] * n - (g.sum(dim=1) / d)[:, None] * (1.0 if layer else 0.0)
    dx *= r[:, None]
    if c["residual"]:
        dx += s["dresidual"].double()
    out = {"dx": dx, "dweight": torch.einsum("md,md->d", dy, n)}
    if c["bias"]:
        out["dbias"] = dy.sum(dim=0)
    return out


def _exact_balance(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    z = s["logits"].double().cpu().numpy()
    ids = s["ids"].cpu().numpy()
    live = np.ones(T, bool) if s["mask"] is None else s["mask"].cpu().numpy()
    n = int(live.sum())
    if c["score"] == "softmax":
        log_p, slope = z - np.logaddexp.reduce(z, axis=1, keepdims=True), np.ones_like(z)
    else:
        log_q = -np.logaddexp(0.0, -z)
        log_p, slope = log_q - np.logaddexp.reduce(log_q, axis=1, keepdims=True), np.exp(-np.logaddexp(0.0, z))
    p = np.exp(log_p)
    count = np.bincount(ids[live].reshape(-1), minlength=E)
    share = p[live].sum(axis=0) / max(n, 1)
    f = count / (max(n, 1) * k)
    out = {"counts": torch.from_numpy(np.append(count, n).astype(np.int32)), "shares": torch.from_numpy(share),
           "loss": torch.tensor([E * float(f @ share)], dtype=torch.float64)}
    if c["back"]:
        a = float(s["dloss"].double()) * E * f / max(n, 1)
        d = np.where(live[:, None], p * (a - (p @ a)[:, None]), 0.0)
        at = np.arange(T)[:, None]
        chosen = log_p[at, ids]
        w = np.exp(chosen - np.logaddexp.reduce(chosen, axis=1, keepdims=True))
        g = s["dweights"].double().cpu().numpy()
        d[at, ids] += w * (g - (w * g).sum(axis=1, keepdims=True))
        out["dlogits"] = torch.from_numpy(d * slope)
    return out


def _exact_rounded(x):
    """Each value of x to the nearest multiple of its block's scale that 4 bits hold, in 64 bits."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    e = torch.frexp(b.abs().amax(dim=-1, keepdim=True))[1] - 1      # floor(log2 of the largest)
    unit = torch.exp2((e - 2).clamp(min=-127).double())
    v = b / unit
    step = torch.where(v.abs() < 2.0, 0.5, torch.where(v.abs() < 4.0, 1.0, 2.0))
    return (torch.clamp(torch.round(v / step) * step, -6.0, 6.0) * unit).reshape(x.shape)   # round: ties to even


def _exact_rounded_t(x):
    return _exact_rounded(torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % 32)).T.contiguous())


def _exact_quantize(s):
    out = {"values": _exact_rounded(s["x"])}
    if s["case"]["both"]:
        out["values_t"] = _exact_rounded_t(s["x"])
    return out


def _exact_values(codes, scales):
    """What packed codes and scales stand for, in 64 bits."""
    nib = torch.stack([codes % 16, codes // 16], dim=2).flatten(1).long()
    man, ex, sign = nib % 2, nib // 2 % 4, 1.0 - 2.0 * (nib // 8)
    mag = torch.where(ex == 0, 0.5 * man, torch.exp2(ex.double() - 1.0) * (1.0 + 0.5 * man))
    rows, K = nib.shape
    block = torch.arange(K, device=codes.device) // 32
    unit = torch.exp2(scales[block // 8, :rows, block % 8].double() - 127.0)   # [K, rows]
    return sign * mag * unit.T


def _exact_gate(name, z):
    if name in ("swiglu", "glu"):
        q = torch.sigmoid(z)
        return z * q if name == "swiglu" else q
    if name in ("gelu_tanh", "geglu"):   # z sigmoid(2 v), v the polynomial inside the tanh
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    r = torch.relu(z)
    return r ** 2 if name == "relu_sq" else r if name in ("relu", "reglu") else z


def _exact_mx4(s):
    c = s["case"]
    if c.get("back"):
        return {"dx": _exact_rounded(s["dy"]) @ _exact_values(s["w"], s["w_scales"]).T,
                "dw": _exact_rounded_t(s["dy"]) @ _exact_rounded_t(s["x"]).T}
    M, N, many = c["M"], c["N"], c["op"] == "experts"
    off = s["offsets"].cpu().tolist() if many else [0, M]
    x = _exact_rounded(s["x"])
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        if a == b:
            continue

        def product(w, scales, bias):
            w, scales = (w[e], scales[e]) if many else (w, scales)
            z = x[a:b] @ _exact_values(w, scales).T
            return z if bias is None else z + (bias[e] if many else bias).double()

        g = _exact_gate(c["act"], product(s["w"], s["w_scales"], s["bias"]))
        y[a:b] = g if s["w_up"] is None else g * product(s["w_up"], s["w_up_scales"], s["bias_up"])
    return {"y": y}
