"""GPU tests of the norm and of the router's balance loss against float64, over sizes and values where they can go
wrong. Bounds count roundings (norm_reference); whole numbers have to be equal."""
import math

import pytest
import torch

import gated_mlp_gemms_amd as gm
import moe_reference as R
import norm_reference as N
from gpu_helpers import announce
from test_gpu_moe import DEV, gen, normal, poison

pytestmark = pytest.mark.gpu
F32 = torch.float32


# ---- norm -----------------------------------------------------------------------------------------

SIZES = [  # rows, widths in 16-byte pieces: around each number of lanes and pieces a lane, and past the registers
    (1, 1), (3, 2), (17, 16), (5, 17), (70, 64), (9, 65), (33, 128), (2, 129), (7, 257), (1030, 100), (1027, 130),
    (1025, 256), (1026, 512), (4, 512), (3, 513), (2, 1024), (5, 1025), (3, 2048), (2, 2049), (1, 5000), (2, 8192),
    (3, 8193), (1, 20001), (5003, 3),
]


def make(g, M, d, dt, wide):
    wt = F32 if wide else dt
    x = (torch.randn(M, d, device=DEV, generator=g) * torch.exp(0.5 * torch.randn(d, device=DEV, generator=g)) + 0.5).to(dt)
    return x, normal(g, M, d, dtype=dt), (1 + 0.2 * normal(g, d)).to(wt), normal(g, d, scale=0.1, dtype=wt)


def check_fwd(x, residual, w, b, kind, eps=1e-5):
    M, d = x.shape
    dt = x.dtype
    y, mean, rstd = poison(M, d, dtype=dt), poison(M, dtype=F32), poison(M, dtype=F32)
    h = poison(M, d, dtype=dt) if residual is not None else None
    gm.norm_fwd(x, y, weight=w, bias=b, residual=residual, h=h, mean=mean if kind == "layer" else None, rstd=rstd, kind=kind, eps=eps)
    kept = N.sum_of(x, residual)
    if residual is not None:
        assert torch.equal(h, (x.float() + residual.float()).to(dt))
        kept = h
    ry, rm, rs, ey, em, es = N.norm_fwd(kept, w, b, kind, eps)
    R.check("rstd", rstd, rs, es + U(rs))
    if kind == "layer":
        R.check("mean", mean, rm, em + U(rm) + R.floor_of(F32))
    R.check("y", y, ry, R.half_step(dt) * ry.abs() + ey * (1 + R.half_step(dt)) + R.floor_of(dt))
    return kept, rm.float() if kind == "layer" else None, rs.float()


def U(v):
    return R.U32 * v.abs()


def check_bwd(dy, h, mean, rstd, w, dres, kind, bias):
    M, d = h.shape
    dt, wt = h.dtype, w.dtype if w is not None else h.dtype
    rx, rw, rb, ex, ew, eb = N.norm_bwd(dy, h, mean, rstd, w, dres, kind)
    dx, dw, db = poison(M, d, dtype=dt), poison(d, dtype=wt), poison(d, dtype=wt) if bias else None
    gm.norm_bwd(dy, h, rstd, dx, mean=mean, weight=w, dresidual=dres, dweight=dw, dbias=db, kind=kind)
    R.check("dx", dx, rx, R.half_step(dt) * rx.abs() + ex * (1 + R.half_step(dt)) + R.floor_of(dt))
    R.check("dweight", dw, rw, R.half_step(wt) * rw.abs() + ew * (1 + R.half_step(wt)) + R.floor_of(wt))
    if bias:
        R.check("dbias", db, rb, R.half_step(wt) * rb.abs() + eb * (1 + R.half_step(wt)) + R.floor_of(wt))
    # added into fp32 buffers, dx in the place of dresidual
    start = normal(gen(1), d, scale=3.0)
    dw2, db2 = start.clone(), start.clone()
    dx2 = dres.clone() if dres is not None else poison(M, d, dtype=dt)
    gm.norm_bwd(dy, h, rstd, dx2, mean=mean, weight=w, dresidual=dx2 if dres is not None else None, dweight=dw2, dbias=db2,
                kind=kind, grad_accum=True)
    assert torch.equal(dx2, dx)
    for name, got, ref, e in (("dweight", dw2, rw, ew), ("dbias", db2, rb, eb)):
        R.check(name + " added", got, ref + start.double(), e + U(ref) + U(ref + start.double()))


@pytest.mark.parametrize("M,pieces", SIZES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm(M, pieces, kind):
    for i, dt in enumerate(R.DT.values()):
        d = pieces * (4 if dt == F32 else 8)
        for wide in ((True,) if dt == F32 else (False, True)):
            announce(f"norm M={M} d={d} {kind} {dt} wide={wide}")
            g = gen(M * 100 + pieces + i)
            x, r, w, b = make(g, M, d, dt, wide)
            b = b if kind == "layer" else None
            check_fwd(x, None, w, b, kind)
            h, mean, rstd = check_fwd(x, r, w, b, kind)
            dy, dres = normal(g, M, d, dtype=dt), normal(g, M, d, dtype=dt)
            check_bwd(dy, h, mean, rstd, w, dres if wide else None, kind, b is not None)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_without_weights_and_with_less_asked_for(kind):
    g, M, d = gen(3), 37, 264
    for dt in R.DT.values():
        x, r, w, _ = make(g, M, d, dt, False)
        h, mean, rstd = check_fwd(x, None, None, None, kind)
        dy = normal(g, M, d, dtype=dt)
        check_bwd(dy, h, mean, rstd, None, None, kind, True)
        whole = [poison(M, d, dtype=dt), poison(d, dtype=dt), poison(d, dtype=dt)]
        gm.norm_bwd(dy, h, rstd, whole[0], mean=mean, weight=w, dweight=whole[1], dbias=whole[2], kind=kind)
        for name, at in (("dx", 0), ("dweight", 1), ("dbias", 2)):
            one = torch.empty_like(whole[at])
            gm.norm_bwd(dy, h, rstd, mean=mean, weight=w, kind=kind, **{name: one})
            assert torch.equal(one, whole[at]), name
        y, y2 = torch.empty_like(x), torch.empty_like(x)
        gm.norm_fwd(x, y, weight=w, residual=r, kind=kind)            # neither the sum nor the statistics kept
        s = x.clone()
        gm.norm_fwd(s, y2, weight=w, residual=r, h=s, kind=kind)      # the sum in x's place
        assert torch.equal(y, y2) and torch.equal(s, (x.float() + r.float()).to(dt))
        s = r.clone()
        gm.norm_fwd(x, y2, weight=w, residual=s, h=s, kind=kind)      # and in the residual's
        assert torch.equal(y, y2) and torch.equal(s, (x.float() + r.float()).to(dt))


@pytest.mark.parametrize("M,d", [(3, 64), (1100, 1024), (2, 4096), (2, 66000)])
def test_norm_of_extreme_rows(M, d):
    """Rows of one value (variance 0), a mean far above the spread, large and tiny values; a NaN or an infinity stays in
    its row."""
    for dt in R.DT.values():
        announce(f"norm extremes {M} {d} {dt}")
        g = gen(d)
        big = 100.0 if dt == torch.float16 else 1e15
        for scale, shift in ((0.0, 3.0), (1.0, 200.0), (big, 0.0), (1e-4, 0.0)):
            x = (torch.randn(M, d, device=DEV, generator=g) * scale + shift).to(dt)
            check_fwd(x, None, torch.ones(d, device=DEV, dtype=dt), None, "layer")
            check_fwd(x, None, None, None, "rms")
        x = normal(g, M, d, dtype=dt)
        y, ref = poison(M, d, dtype=dt), poison(M, d, dtype=dt)
        gm.norm_fwd(x, ref)
        for v in (math.nan, math.inf, -math.inf):
            z = x.clone()
            z[1, d // 2] = v
            gm.norm_fwd(z, y)
            assert torch.isnan(y[1]).all()
            keep = [i for i in range(M) if i != 1]
            assert torch.equal(y[keep], ref[keep])


def test_norm_of_no_rows():
    for dt in R.DT.values():
        x, w = torch.empty(0, 64, dtype=dt, device=DEV), torch.ones(64, dtype=dt, device=DEV)
        gm.norm_fwd(x, torch.empty_like(x), weight=w, mean=torch.empty(0, device=DEV), rstd=torch.empty(0, device=DEV))
        dw, db, kept = poison(64, dtype=dt), poison(64, dtype=dt), torch.full((64,), 2.5, device=DEV)
        stat = torch.empty(0, device=DEV)
        gm.norm_bwd(x, x, stat, torch.empty_like(x), mean=stat, weight=w, dweight=dw, dbias=db)
        assert not dw.any() and not db.any()
        gm.norm_bwd(x, x, stat, torch.empty_like(x), mean=stat, weight=w, dweight=kept, grad_accum=True)
        assert (kept == 2.5).all()


def test_norm_gradient_is_a_difference():
    """fp32 gradients against central differences of the float64 formula, over rows of every kernel."""
    for M, d, kind in ((6, 40, "layer"), (5, 2052, "rms"), (3, 8200, "layer"), (2, 40000, "layer")):
        announce(f"norm differences {M} {d} {kind}")
        g = gen(d)
        x, r, w, b = make(g, M, d, F32, True)
        dy = normal(g, M, d)
        y, h, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(M, device=DEV), torch.empty(M, device=DEV)
        mean = mean if kind == "layer" else None
        gm.norm_fwd(x, y, weight=w, bias=b, residual=r, h=h, mean=mean, rstd=rstd, kind=kind)
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        gm.norm_bwd(dy, h, rstd, dx, mean=mean, weight=w, dweight=dw, dbias=db, kind=kind)

        def loss(h, w, b):
            return (N.norm_fwd(h, w, b, kind, 1e-5)[0] * dy.double()).sum()

        at, step = [h.double(), w.double(), b.double()], 1e-5
        for i, grad in enumerate((dx, dw, db)):
            v = torch.randn(at[i].shape, device=DEV, generator=g, dtype=torch.float64)
            hi, lo = ([a + s * step * v if j == i else a for j, a in enumerate(at)] for s in (1, -1))
            diff = (loss(*hi) - loss(*lo)) / (2 * step)
            scale = (grad.double().abs() * v.abs()).sum()
            # the statistics are fp32 values here and exact there: their half steps, of every factor, on top
            assert abs(diff - (grad.double() * v).sum()) <= 400 * R.U32 * scale + 1e-6 * scale


def test_norm_same_bits_again_on_another_stream_and_in_a_graph():
    for M, d in ((300, 1032), (2000, 4096), (3, 17000)):
        g, dt = gen(d), torch.bfloat16
        x, r, w, b = make(g, M, d, dt, True)
        dy = normal(g, M, d, dtype=dt)
        out = dict(y=torch.empty_like(x), h=torch.empty_like(x), mean=torch.empty(M, device=DEV), rstd=torch.empty(M, device=DEV),
                   dx=torch.empty_like(x), dw=torch.empty_like(w), db=torch.empty_like(b))

        def step(stream=None, ws=torch.empty(gm.norm_workspace_bytes(M, d), dtype=torch.uint8, device=DEV)):
            gm.norm_fwd(x, out["y"], weight=w, bias=b, residual=r, h=out["h"], mean=out["mean"], rstd=out["rstd"], stream=stream)
            gm.norm_bwd(dy, out["h"], out["rstd"], out["dx"], mean=out["mean"], weight=w, dresidual=dy, dweight=out["dw"],
                        dbias=out["db"], workspace=ws, stream=stream)

        step()
        torch.cuda.synchronize()
        first = {n: t.clone() for n, t in out.items()}
        side = torch.cuda.Stream()
        for stream in (None, side, side.cuda_stream):
            for t in out.values():
                t.zero_()
            torch.cuda.synchronize()
            step(stream)
            torch.cuda.synchronize()
            assert all(torch.equal(first[n], t) for n, t in out.items())
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            step()
        for i in range(3):
            x.copy_(normal(gen(i), M, d, dtype=dt))
            graph.replay()
            torch.cuda.synchronize()
            replayed = {n: t.clone() for n, t in out.items()}
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(replayed[n], t) for n, t in out.items())


# ---- balance loss -----------------------------------------------------------------------------------

BALANCE = [  # T, E, k
    (1, 1, 1), (1, 7, 2), (3, 16, 16), (31, 17, 4), (65, 60, 3), (1000, 64, 4), (333, 128, 8), (40, 129, 6), (257, 256, 8),
    (50, 500, 8), (9, 1024, 16), (5000, 33, 5), (20000, 8, 2),
]


def run_balance(x, ids, mask, score):
    T, E = x.shape
    counts, shares, loss = poison(E + 1, dtype=torch.int32), poison(E, dtype=F32), poison(1, dtype=F32)
    gm.moe_balance(x, ids, counts, shares, loss, mask=mask, score=score)
    return counts, shares, loss


def check_balance(x, ids, mask, score, g):
    T, E = x.shape
    k = ids.shape[1]
    counts, shares, loss = run_balance(x, ids, mask, score)
    rc, rp, rl = N.balance(x, ids, mask, score)
    assert torch.equal(counts.long(), rc)
    # a probability is a ratio of a sum of E exponentials, each off by its argument's rounding; shares sum over the
    # tokens, a group's one after another, then the groups, the waves and the parts
    live = torch.nan_to_num(x.double() if mask is None else x.double()[mask], neginf=0.0, posinf=0.0)
    span = live.abs().max().item() if live.numel() else 0.0
    rel = (E + 32 + 4 * span) * R.U32
    deep = rel + (T / 128 + 200) * R.U32
    R.check("shares", shares, rp, deep * rp + 1e-37)
    R.check("loss", loss, rl.reshape(1), ((E + deep / R.U32) * R.U32 * rl).reshape(1) + 1e-37)
    dloss = torch.tensor([0.7], device=DEV)
    dw = normal(g, T, k, scale=1.0 / T)
    for weights, renorm in ((None, True), (dw, True), (dw, False)):
        dl = poison(T, E, dtype=x.dtype)
        gm.moe_balance_bwd(x, ids, counts, dl, mask=mask, dloss=dloss, dweights=weights, score=score, renorm=renorm)
        ref, size = N.balance_bwd(x, counts, k, mask, dloss.double().item(), score)
        mag = torch.zeros_like(ref)
        if weights is not None:
            route = R.route_bwd(x, ids.long(), weights, score, renorm)
            ref = ref + route
            p = N.probs(x, score)[0] if score == "softmax" else torch.sigmoid(x.double())
            pw = p.gather(1, ids.long())
            pw = pw / torch.where(pw.sum(1, keepdim=True) == 0, 1.0, pw.sum(1, keepdim=True)) if renorm else pw
            mag = 2 * rel * ((weights.double().abs() * pw).sum(dim=1, keepdim=True) * 2 + weights.abs().max())
        bound = R.half_step(x.dtype) * ref.abs() + (4 * rel + (E + 8) * R.U32) * size + mag + R.floor_of(x.dtype)
        R.check("dlogits", dl, ref, bound)
    # without a loss' gradient of its own it is the loss'
    one, none = poison(T, E, dtype=x.dtype), poison(T, E, dtype=x.dtype)
    gm.moe_balance_bwd(x, ids, counts, one, mask=mask, dloss=torch.ones(1, device=DEV), score=score)
    gm.moe_balance_bwd(x, ids, counts, none, mask=mask, score=score)
    assert torch.equal(one, none)


@pytest.mark.parametrize("T,E,k", BALANCE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance(T, E, k, score):
    for i, dt in enumerate(R.DT.values()):
        announce(f"balance T={T} E={E} k={k} {score} {dt}")
        g = gen(T + E * 1000 + i)
        x = normal(g, T, E, scale=2.0, dtype=dt)
        ids, _ = R.route(x, k, score, True)[:2]
        ids = ids.int().contiguous()
        check_balance(x, ids, None, score, g)
        check_balance(x, ids, torch.rand(T, device=DEV, generator=g) < 0.6, score, g)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_of_extremes(score):
    for dt in R.DT.values():
        g = gen(11)
        x = normal(g, 64, 70, dtype=dt)
        x[3] = -math.inf                                   # a token without any expert
        x[4, 1:] = -math.inf
        x[6] = torch.finfo(torch.float16).min
        x[7, 3] = 60000.0
        x[8] = -80.0
        ids = R.route(x, 6, score, True)[0].int().contiguous()
        check_balance(x, ids, None, score, g)
        # what tokens that do not count hold does not matter, nor do ids out of range
        mask = torch.ones(64, dtype=torch.bool, device=DEV)
        mask[10:20] = False
        counts, shares, loss = run_balance(x, ids, mask, score)
        y, some = x.clone(), ids.clone()
        y[10], y[11], y[12, 5] = math.nan, math.inf, -math.inf
        some[13] = -7
        for a, b in zip(run_balance(y, some, mask, score), (counts, shares, loss)):
            assert torch.equal(a, b)
        dl, ref = poison(64, 70, dtype=dt), poison(64, 70, dtype=dt)
        gm.moe_balance_bwd(y, some, counts, dl, mask=mask, score=score)
        gm.moe_balance_bwd(x, ids, counts, ref, mask=mask, score=score)
        assert torch.equal(dl, ref) and not dl[10:20].any()
        some = ids.clone()
        some[20, 2], some[21] = 70, -1
        assert torch.equal(run_balance(x, some, None, score)[0].long(), N.balance(x, some, None, score)[0])


def test_balance_of_nothing():
    for T in (0, 5):
        x, ids = torch.randn(T, 12, device=DEV), torch.zeros(T, 2, dtype=torch.int32, device=DEV)
        mask = torch.zeros(T, dtype=torch.bool, device=DEV)
        counts, shares, loss = run_balance(x, ids, mask, "softmax")
        assert not counts.any() and not shares.any() and float(loss) == 0.0
        dl = poison(T, 12, dtype=F32)
        gm.moe_balance_bwd(x, ids, counts, dl, mask=mask)
        assert not dl.any()


def test_balance_nan_is_seen():
    x, ids = normal(gen(1), 40, 20), torch.zeros(40, 2, dtype=torch.int32, device=DEV)
    x[17, 3] = math.nan
    counts, shares, loss = run_balance(x, ids, None, "softmax")
    assert torch.isnan(loss).all() and int(counts[0]) == 80


def test_balance_even_load_is_one():
    """k choices spread evenly and equal scores: the loss is 1, whatever T, E and k."""
    for T, E, k in ((48, 16, 4), (60, 60, 3)):
        ids = (torch.arange(T * k, device=DEV, dtype=torch.int32) % E).reshape(T, k)
        for score in ("softmax", "sigmoid"):
            loss = run_balance(torch.full((T, E), 0.3, device=DEV), ids, None, score)[2]
            assert abs(float(loss) - 1.0) <= (E + 64) * R.U32


def test_balance_gradient_is_a_difference():
    g = gen(4)
    for score in ("softmax", "sigmoid"):
        x = normal(g, 50, 24)
        ids = R.route(x, 3, score, True)[0].int().contiguous()
        mask = torch.rand(50, device=DEV, generator=g) < 0.8
        counts, _, _ = run_balance(x, ids, mask, score)
        dl = poison(50, 24, dtype=F32)
        gm.moe_balance_bwd(x, ids, counts, dl, mask=mask, score=score)
        v = torch.randn(50, 24, device=DEV, generator=g, dtype=torch.float64)
        hi, lo = (N.balance(x.double() + s * 1e-5 * v, ids, mask, score)[2] for s in (1, -1))
        scale = (dl.double().abs() * v.abs()).sum()
        assert abs((hi - lo) / 2e-5 - (dl.double() * v).sum()) <= 200 * R.U32 * scale + 1e-6 * scale


def test_balance_same_bits_again_on_another_stream_and_in_a_graph():
    g = gen(8)
    T, E, k = 3000, 60, 4
    x = normal(g, T, E, dtype=torch.bfloat16)
    ids = R.route(x, k, "softmax", True)[0].int().contiguous()
    mask = torch.rand(T, device=DEV, generator=g) < 0.9
    out = dict(counts=poison(E + 1, dtype=torch.int32), shares=poison(E, dtype=F32), loss=poison(1, dtype=F32),
               dl=poison(T, E, dtype=torch.bfloat16))
    dw = normal(g, T, k, scale=1.0 / T)

    def step(stream=None):
        gm.moe_balance(x, ids, out["counts"], out["shares"], out["loss"], mask=mask, stream=stream)
        gm.moe_balance_bwd(x, ids, out["counts"], out["dl"], mask=mask, dweights=dw, stream=stream)

    step()
    torch.cuda.synchronize()
    first = {n: t.clone() for n, t in out.items()}
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        for t in out.values():
            t.zero_()
        torch.cuda.synchronize()
        step(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(first[n], t) for n, t in out.items())
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        x.copy_(normal(gen(i), T, E, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        replayed = {n: t.clone() for n, t in out.items()}
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(replayed[n], t) for n, t in out.items())
