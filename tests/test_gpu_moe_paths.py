"""GPU tests of the mixture-of-experts operators on the paths that their main tests do not take."""
import pytest
import torch

import gated_mlp_gemms_amd as gm
import moe_paths as P
import moe_reference as R
from gpu_helpers import announce
from test_gpu_moe import DEV, check_linear, gen, normal, offsets_of, poison

pytestmark = pytest.mark.gpu


# ---- streams ------------------------------------------------------------------------------------

def test_workspaces_of_calls_on_a_stream_that_is_passed():
    """Without a workspace, on a stream that is not torch's current one: the same bits, and the memory that the
    call allocates belongs to its stream."""
    g, dt = gen(32), torch.bfloat16
    T, E, k, d, h = 2100, 6, 3, 264, 520
    n = T * k
    ids = torch.rand(T, E, device=DEV, generator=g).topk(k, dim=1)[1].to(torch.int32)
    x, dy, w, b = normal(g, n, d, dtype=dt), normal(g, n, h, dtype=dt), normal(g, E, h, d, scale=0.05, dtype=dt), normal(g, E, h, dtype=dt)
    experts = gm.make_linear_desc(n, d, h, act="gelu_tanh", dtype=dt, experts=E)
    deep = gm.make_linear_desc(130, 8200, 264, dtype=dt)        # split along K into partial sums
    xd, wd = normal(g, 130, 8200, dtype=dt), normal(g, 264, 8200, scale=0.01, dtype=dt)
    mlp = gm.make_desc(300, d, h, act="swiglu", dtype=dt)
    xm, wg, wu, wo = normal(g, 300, d, dtype=dt), w[0].contiguous(), w[1].contiguous(), normal(g, d, h, scale=0.05, dtype=dt)
    assert n > 4096 and gm.linear_workspace_bytes(deep, "fwd") > 256   # (the sort counts in its workspace)

    def run(stream):
        off, row, slot = (poison(m, dtype=torch.int32) for m in (E + 1, n, n))
        y, pre, yd, ym = (poison(*s, dtype=dt) for s in ((n, h), (n, h), (130, 264), (300, d)))
        dx, dw, db = poison(n, d, dtype=dt), poison(E, h, d, dtype=dt), poison(E, h, dtype=dt)
        torch.cuda.synchronize()
        gm.moe_sort(ids, E, off, row, slot, stream=stream)
        gm.linear_fwd(experts, x, w, y, bias=b, offsets=off, preact=pre, stream=stream)
        gm.linear_bwd(experts, dy, x, w, preact=pre, offsets=off, dx=dx, dw=dw, dbias=db, stream=stream)
        gm.linear_fwd(deep, xd, wd, yd, stream=stream)
        gm.mlp_fwd_infer(mlp, xm, wg, wu, wo, ym, stream=stream)
        torch.cuda.synchronize()
        return off, row, slot, y, pre, dx, dw, db, yd, ym

    first = run(None)
    for handle in (False, True):
        side = torch.cuda.Stream()
        assert side.cuda_stream != torch.cuda.current_stream().cuda_stream
        announce(f"workspaces on {side}")
        assert all(torch.equal(a, c) for a, c in zip(first, run(side.cuda_stream if handle else side)))
        held = sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == side.cuda_stream)
        assert held >= gm.linear_workspace_bytes(experts, "bwd")


# ---- router -------------------------------------------------------------------------------------

def route_both(x, k, renorm, g):
    """ids, weights, dweights and dlogits of a sigmoid router."""
    T, E = x.shape
    ids, w, dw = poison(T, k, dtype=torch.int32), poison(T, k, dtype=torch.float32), normal(g, T, k)
    dl = poison(T, E, dtype=x.dtype)
    gm.moe_route(x, ids, w, score="sigmoid", renorm=renorm)
    gm.moe_route_bwd(x, ids, dw, dl, score="sigmoid", renorm=renorm)
    return ids.long(), w, dw, dl


def sigmoid_reference(x, ids, dw, renorm):
    """In float64, from the logarithms so that nothing underflows or cancels: weights, dlogits at the chosen experts and
    what the latter's error counts by (|w| (1 - q) times the terms of g - mean; unnormalised: the value)."""
    s, g = x.double().gather(1, ids), dw.double()
    logq, rest = torch.nn.functional.logsigmoid(s), torch.sigmoid(-s)
    if not renorm:
        return logq.exp(), logq.exp() * rest * g, (logq.exp() * rest * g).abs()
    w = torch.softmax(logq, dim=1)
    mean = (g * w).sum(dim=1, keepdim=True)
    return w, w * rest * (g - mean), w * rest * (g.abs() + (g.abs() * w).sum(dim=1, keepdim=True))


@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_far_from_zero(renorm):
    """Scores up to 30, whose sigmoids are 1 in fp32 and their gradients are not 0: the error is a few roundings of the
    value itself. The exponential is off by 2 half steps at most, 1 + t, its reciprocal, two products and the last
    by one each: 8; a normalised weight adds its total's (k + 8) and a quotient's, twice (in w and in the mean)."""
    k = 8
    for dt in R.DT.values():
        announce(f"sigmoid gradient renorm={renorm} {dt}")
        g = gen(60)
        x = (torch.linspace(-30, 30, 320, device=DEV)[torch.randperm(320, device=DEV, generator=g)]).reshape(8, 40).to(dt)
        ids, w, dw, dl = route_both(x, k, renorm, g)
        rw, rd, mag = sigmoid_reference(x, ids, dw, renorm)
        n = 8 + 2 * (k + 10) if renorm else 8
        R.check("dlogits", dl.gather(1, ids), rd, n * R.U32 * mag + R.half_step(dt) * rd.abs() + R.floor_of(dt))


def test_sigmoid_weights_of_low_scores():
    """Scores whose sigmoids leave fp32's range (below -88): normalised, they are the weights of any other scores; the
    sigmoid itself is as near as fp32 has it. The bound counts as above, the exponential of a difference of scores a
    half step of the difference more."""
    k = 6
    for dt in (torch.float32, torch.bfloat16):
        announce(f"sigmoid weights of low scores {dt}")
        g = gen(61)
        low = -20.0 - 83.0 * torch.rand(40, 24, device=DEV, generator=g)
        low[0], low[1], low[2, 5:] = -95.0, -103.0, -200.0
        low[3] = torch.linspace(-102, -88, 24, device=DEV)
        low[4, 0] = 3.0                                    # a score of ordinary size among them
        x = low.to(dt)
        ids, w, dw, dl = route_both(x, k, True, g)
        rw, rd, mag = sigmoid_reference(x, ids, dw, True)
        s = x.double().gather(1, ids)
        n = 2 * (k + 18) + 2 * (s[:, :1] - s)
        tiny = 2 * torch.finfo(torch.float32).smallest_normal      # weights below fp32's range, and what they enter
        R.check("weights", w, rw, n * R.U32 * rw + tiny)
        R.check("dlogits", dl.gather(1, ids), rd,
                n * R.U32 * mag + tiny * (1 + dw.abs().max().item()) * k + R.half_step(dt) * rd.abs() + R.floor_of(dt))
        x[:] = -105.0                                      # below 2^-150 all of them count as 0
        _, w, _, dl = route_both(x, k, True, g)
        assert not w.any() and not dl.any()
        x[:] = torch.linspace(-100, -70, 24, device=DEV)
        ids, w, _, _ = route_both(x, k, False, g)
        ref = torch.sigmoid(x.double().gather(1, ids))
        R.check("weights", w, ref, 8 * R.U32 * ref + 2 * R.floor_of(torch.float32))


# ---- activations --------------------------------------------------------------------------------

def slopes(act, z, u=1.0):
    """f'(z) and, gated, f(z) as linear_bwd forms them, in fp32: the bias gradients of one row against dy = 1."""
    N, dt, gated = z.numel(), z.dtype, act in R.GATED
    desc = gm.make_linear_desc(1, 8, N, act=act, dtype=dt)
    pre = (torch.cat([z, torch.full_like(z, u)]) if gated else z).reshape(1, -1).contiguous()
    x, w, dy = (torch.ones(*s, dtype=dt, device=DEV) for s in ((1, 8), (N, 8), (1, N)))
    db, du = torch.zeros(N, device=DEV), torch.zeros(N, device=DEV)
    gm.linear_bwd(desc, dy, x, w, w_up=w if gated else None, preact=pre, dbias=db, dbias_up=du if gated else None,
                  grad_accum=True)
    return db, du


@pytest.mark.parametrize("dtype", list(R.DT))
def test_glu_gradient_far_from_zero(dtype):
    """Gates up to 80, where the sigmoid is 1 in fp32 and its gradient is not 0. Its exponential is off by |z| + 2 half
    steps (fp32's argument), 1 + e, the reciprocal (2), two products by 6 in all; each counts in s, in s and in e."""
    z = torch.linspace(-80, 80, 400, device=DEV).to(R.DT[dtype])
    df, f = slopes("glu", z)
    s = torch.sigmoid(z.double())
    ref = s * torch.sigmoid(-z.double())
    n = 3 * (z.double().abs() + 8)
    R.check("f", f, s, n * R.U32 * s)
    R.check("df", df, ref, n * R.U32 * ref)


@pytest.mark.parametrize("act", [a for a in R.ACTS if a != "none"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slopes_of_large_values(act, dtype):
    """From 1e5 to 1e38 every f' has reached its limit: 1, 0 or, of relu^2, 2 z."""
    z = torch.tensor([s * 10.0 ** e for e in (5, 7, 9, 13, 17, 18, 19, 20, 25, 30, 33, 38) for s in (1, -1)], device=DEV).to(R.DT[dtype])
    df, _ = slopes(act, z)
    up = {"glu": 0.0, "relu_sq": 2 * z.float().clamp(min=0)}.get(act, (z > 0).float())
    assert torch.equal(df, torch.broadcast_to(torch.as_tensor(up, device=DEV), df.shape))


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("M", [3, 100, 700])     # streamed, and in small and large tiles
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_comes_through(act, M, dtype):
    """A NaN in one row of x makes that row of y NaN, of every activation, and no other."""
    dt, g, gated = R.DT[dtype], gen(62), act in R.GATED
    K, N = 72, 1032
    x, w, u = normal(g, M, K, dtype=dt), normal(g, N, K, dtype=dt), normal(g, N, K, dtype=dt) if gated else None
    x[1, 5] = float("nan")
    for experts, off in ((0, None), (1, offsets_of([M]))):
        desc = gm.make_linear_desc(M, K, N, act=act, dtype=dt, experts=experts)
        lead = (lambda t: t[None] if experts and t is not None else t)
        y, pre = torch.zeros(M, N, dtype=dt, device=DEV), torch.zeros(M, 2 * N if gated else N, dtype=dt, device=DEV)
        gm.linear_fwd(desc, x, lead(w), y, w_up=lead(u), offsets=off, preact=pre)
        assert torch.isnan(y[1]).all() and torch.isnan(pre[1]).all()
        rest = torch.arange(M, device=DEV) != 1
        assert torch.isfinite(y[rest]).all() and torch.isfinite(pre[rest]).all()


# ---- rows ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,d,dtype", [(2100, 4096, "bf16"), (1500, 4096, "f16"), (2200, 2060, "f32")])
def test_streamed_rows_equal_rows_in_caches(T, d, dtype):
    """From 32 MiB of sorted rows on they are streamed: the same values as of the tokens in eight parts, which are not."""
    g, dt, E, k, parts = gen(22), R.DT[dtype], 24, 3, 8
    n, size = T * k, torch.empty(0, dtype=dt).element_size()
    assert n * d * size >= 32 << 20 and -(-T // parts) * k * d * size < 16 << 20
    ids = torch.rand(T, E, device=DEV, generator=g).topk(k, dim=1)[1].to(torch.int32)
    ids[torch.rand(T, k, device=DEV, generator=g) < 0.1] = -1
    x, dout, w = normal(g, T, d, dtype=dt), normal(g, T, d, dtype=dt), torch.rand(T, k, device=DEV, generator=g)
    each = normal(g, n, d, dtype=dt)               # a row of ys for each slot

    def layer(a, b):
        m = (b - a) * k
        off, row, slot = (poison(c, dtype=torch.int32) for c in (E + 1, m, m))
        gm.moe_sort(ids[a:b].contiguous(), E, off, row, slot)
        ys = each[a * k:b * k][slot.long()]
        xs, out, dys, dw, dx = (poison(*s, dtype=t) for s, t in (
            ((m, d), dt), ((b - a, d), dt), ((m, d), dt), ((b - a, k), torch.float32), ((b - a, d), dt)))
        gm.moe_gather(x[a:b].contiguous(), slot, off, xs)
        gm.moe_combine(ys, w[a:b].contiguous(), row, off, out, residual=x[a:b].contiguous())
        gm.moe_combine_bwd(dout[a:b].contiguous(), ys, w[a:b].contiguous(), row, slot, off, dys, dw)
        gm.moe_gather_bwd(ys, row, off, dx)
        at = row.long()                            # by slot again
        return xs[at], out, dys[at], dw, dx

    cuts = [T * i // parts for i in range(parts + 1)]
    whole, pieces = layer(0, T), [layer(a, b) for a, b in zip(cuts, cuts[1:])]
    for i, t in enumerate(whole):
        assert torch.equal(t, torch.cat([p[i] for p in pieces])), i


# ---- every kernel of the products ---------------------------------------------------------------

@pytest.mark.parametrize("p", P.PATHS, ids=lambda p: f"{p.M}x{p.K}x{p.N}-{p.act}-{p.dtype}-{len(p.counts or ())}")
def test_products(p):
    """Forward and backward, with bias and residual."""
    counts = p.counts and list(p.counts)
    check_linear(p.M, p.K, p.N, p.act, R.DT[p.dtype], experts=len(counts or ()), offsets=offsets_of(counts) if counts else None)


@pytest.mark.parametrize("E", [255, 256, 257, 319, 320, 321])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_numbers_of_experts_around_the_searchs(E, dtype):
    """The search for a workgroup's rows holds 1, 4 or 17 experts a lane: up to 64, up to 256, above (one less where the
    rows behind the last offset count). In 16 bits few rows are streamed, many in tiles; in fp32 all in tiles."""
    g = torch.Generator().manual_seed(E)
    for most in (3, 20):
        counts = [int(c) for c in torch.randint(0, most, (E - 2,), generator=g)] + [0, 5]
        check_linear(sum(counts) + 3, 40, 24, "swiglu", R.DT[dtype], experts=E, offsets=offsets_of(counts))
        check_linear(sum(counts), 40, 24, "none", R.DT[dtype], experts=E, offsets=offsets_of(counts))


# streaming (at most 8 rows an expert on average), experts of more than 16 rows among them
CROWDED = [  # rows an expert, rows behind them, K, N
    ([0, 0, 64, 0, 0, 0, 0, 0], 0, 264, 136), ([61, 0, 0, 0, 0, 0, 0, 0], 3, 136, 40), ([0] * 7 + [17], 30, 520, 24),
    ([16, 33, 1, 40, 0, 15, 0, 0, 0, 0, 0, 0, 0, 0, 0, 17], 5, 2056, 72), ([1] * 60 + [130] + [0] * 39 + [200], 40, 136, 264),
    ([0] * 200 + [900, 16, 17, 0, 32, 33] + [2] * 114, 50, 72, 40), ([0] * 1023 + [1500], 1, 40, 24),
]


@pytest.mark.parametrize("case", CROWDED, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[2]}-{c[3]}")
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_streamed_experts_of_many_rows(case, dtype):
    counts, tail, K, N = case
    assert sum(counts) + tail <= 8 * len(counts)
    for act in ("none", "swiglu"):
        check_linear(sum(counts) + tail, K, N, act, R.DT[dtype], experts=len(counts), offsets=offsets_of(counts))


@pytest.mark.parametrize("p", [p for p in P.PATHS if p.counts], ids=lambda p: f"{p.M}x{p.K}x{p.N}-{p.act}-{p.dtype}-{len(p.counts)}")
def test_an_experts_nan_stays_its_own(p):
    """Rows of one expert that are NaN reach no other expert's rows or gradients."""
    dt, g, gated, E = R.DT[p.dtype], gen(63), p.act in R.GATED, len(p.counts)
    announce(f"an expert's NaN {p}")
    off = offsets_of(list(p.counts))
    x, w, dy = normal(g, p.M, p.K, dtype=dt), normal(g, E, p.N, p.K, scale=0.05, dtype=dt), normal(g, p.M, p.N, dtype=dt)
    u = normal(g, E, p.N, p.K, scale=0.05, dtype=dt) if gated else None
    bad = max(e for e in range(E - 1) if p.counts[e])      # one with an expert behind it
    lo, hi = int(off[bad]), int(off[bad + 1])
    x[lo:hi], dy[lo:hi] = float("nan"), float("nan")
    desc = gm.make_linear_desc(p.M, p.K, p.N, act=p.act, dtype=dt, experts=E)
    y, pre, dx = (poison(p.M, n, dtype=dt) for n in (p.N, 2 * p.N if gated else p.N, p.K))
    gm.linear_fwd(desc, x, w, y, w_up=u, offsets=off, preact=pre)
    dw, db = poison(E, p.N, p.K, dtype=dt), poison(E, p.N, dtype=dt)
    dwu, dbu = (torch.zeros_like(dw), torch.zeros_like(db)) if gated else (None, None)
    gm.linear_bwd(desc, dy, x, w, w_up=u, preact=None if p.act == "none" else pre, offsets=off, dx=dx, dw=dw, dw_up=dwu,
                  dbias=db, dbias_up=dbu)
    rows = torch.ones(p.M, dtype=torch.bool, device=DEV)
    rows[lo:hi] = False
    for t in (y, pre, dx):
        assert torch.isfinite(t[rows]).all() and torch.isnan(t[lo:hi]).any()
    others = torch.arange(E, device=DEV) != bad
    for t in filter(lambda t: t is not None, (dw, dwu, db, dbu)):
        assert torch.isfinite(t[others]).all() and torch.isnan(t[bad]).any()


# ---- the layer's runner -------------------------------------------------------------------------

@pytest.mark.parametrize("experts", [8, 7])
def test_runner_sums_dx_in_fp32(experts):
    """dx of a 16-bit layer: the experts' rows summed in fp32 onto dout plus the router's part, and rounded once."""
    from gated_mlp_gemms_amd.moe_runner import MoeRunner, moe_tensors

    size = dict(act="swiglu", dtype="bf16", tokens=70, width=136, hidden=72, experts=experts)
    r = MoeRunner(choices=5, tensors=moe_tensors(seed=7, **size), **size)
    r.step()
    base = (r.dx_router.float() + r.dout.float()).bfloat16().float()
    row, acc = r.row_of.long().reshape(70, 5), torch.zeros(70, 136, device=DEV)
    for j in range(5):
        acc = acc + r.dxs.float()[row[:, j]]
    assert torch.equal(r.dx, (acc + base).bfloat16())


def test_runner_with_a_residual_of_its_own():
    """A norm in front: x is the norm of the stream h, which the output is added to. fp32, against autograd of the formula
    in float64 on the CPU, through the norm; the bound is test_gpu_moe.py's, for one more product's depth."""
    from gated_mlp_gemms_amd.moe_runner import MoeRunner, moe_tensors

    size = dict(act="swiglu", dtype="f32", tokens=45, width=32, hidden=40, experts=8)
    t, h = moe_tensors(seed=8, **size), normal(gen(9), 45, 32)
    norm = lambda h: h / (h.square().mean(dim=1, keepdim=True) + 1e-5).sqrt()   # noqa: E731
    t.update(x=norm(h.double()).float(), residual=h)
    r = MoeRunner(choices=3, tensors=t, **size)
    r.step()
    leaf = {k: t[k].double().cpu().requires_grad_() for k in ("residual", "router", "w_gate", "w_up", "w_down")}
    x, ids = norm(leaf["residual"]), r.ids.long().cpu()
    x.retain_grad()
    w = torch.softmax((x @ leaf["router"].T).gather(1, ids), dim=1)
    out = leaf["residual"]
    for j in range(3):
        e = ids[:, j]
        g, u = ((leaf[n][e] @ x[:, :, None])[:, :, 0] for n in ("w_gate", "w_up"))
        out = out + w[:, j:j + 1] * (leaf["w_down"][e] @ (torch.nn.functional.silu(g) * u)[:, :, None])[:, :, 0]
    (out * t["dout"].double().cpu()).sum().backward()
    grads = r.grads()
    pairs = [("out", r.out, out.detach()), ("dx", grads["dx"], x.grad), ("d_router", grads["d_router"], leaf["router"].grad),
             ("dw1", grads["dw1"], leaf["w_gate"].grad), ("dw_up", grads["dw_up"], leaf["w_up"].grad),
             ("dw2", grads["dw2"], leaf["w_down"].grad)]
    for name, a, b in pairs:
        R.check(name, a.cpu(), b, torch.full_like(b, 2400 * R.U32 * b.abs().max().item()))
    assert torch.equal(MoeRunner(choices=3, tensors=t, train=False, **size).forward_infer(), r.out)
