"""GPU tests of tensors whose offsets pass 32 bits: a small problem's rows (or experts) repeated, so that every
repetition has to be the small problem's result."""
import pytest
import torch

import gated_mlp_gemms_amd as gm
import moe_reference as R
import norm_reference as N
from gpu_helpers import announce
from test_gpu_moe import DEV, gen, normal, offsets_of
from test_gpu_mx4 import check_product

pytestmark = pytest.mark.gpu
U8, BF = torch.uint8, torch.bfloat16


def again(base, reps):
    """base's rows `reps` times."""
    return base.expand(reps, *base.shape).reshape(reps * base.shape[0], *base.shape[1:]).contiguous()


def is_again(t, base):
    return torch.equal(t.reshape(-1, *base.shape), base.expand(t.shape[0] // base.shape[0], *base.shape))


def blocks(rows, K, batch=None):
    return [torch.full(s, 0xEE, dtype=U8, device=DEV) for s in gm.mx4_shapes(rows, K, batch)]


def test_blocks_there_and_back():
    reps, n, K = 8200, 64, 4160
    announce(f"mx4 blocks {reps * n} x {K}")
    base = normal(gen(1), n, K, dtype=BF)
    a, t = blocks(n, K), blocks(K, n)
    gm.mx4_quantize(base, *a, codes_t=t[0], scales_t=t[1])
    x, rows = again(base, reps), reps * n
    assert x.numel() > 1 << 31
    for both in (True, False):
        p, q = blocks(rows, K), blocks(K, rows)
        if both:
            gm.mx4_quantize(x, *p, codes_t=q[0], scales_t=q[1])
        else:
            gm.mx4_quantize(x, *p)
            gm.mx4_quantize(x, None, None, codes_t=q[0], scales_t=q[1])
        assert is_again(p[0], a[0])
        assert all(is_again(p[1][i, :rows], a[1][i, :n]) for i in range(a[1].shape[0]))
        assert (q[0].reshape(K, reps, n // 2) == t[0][:, None]).all()
        assert (q[1][:, :K].transpose(0, 1).reshape(K, -1)[:, : reps * 2].reshape(K, reps, 2) == t[1][0, :K, None, :2]).all()
    del q
    small = torch.empty_like(base)
    gm.mx4_dequantize(*a, small)
    gm.mx4_dequantize(*p, x)
    assert is_again(x, small)


def test_product_of_many_rows():
    reps, n, K, cols = 8200, 256, 4096, 1032
    announce(f"mx4 product {reps * n} x {K} x {cols}")
    g = gen(2)
    (xq, xs), (wq, ws) = ([torch.randint(0, 256, blk.shape, device=DEV, generator=g).to(U8) if i == 0 else
                           torch.randint(120, 130, blk.shape, device=DEV, generator=g).to(U8) for i, blk in enumerate(blocks(r, K))]
                          for r in (n, cols))
    small = torch.empty(n, cols, dtype=BF, device=DEV)
    gm.mx4_linear_fwd(gm.make_linear_desc(n, K, cols, dtype=BF), xq, xs, wq, ws, small)
    M = reps * n
    far = blocks(M, K)
    far[0] = again(xq, reps)
    for i in range(xs.shape[0]):
        far[1][i, :M] = again(xs[i, :n], reps)
    y = torch.empty(M, cols, dtype=BF, device=DEV)
    assert far[0].numel() > 1 << 32 and y.numel() > 1 << 31
    gm.mx4_linear_fwd(gm.make_linear_desc(M, K, cols, dtype=BF), *far, wq, ws, y)
    # another tile, another order of the sums: both are within a rounding of each other
    ref = small.double()
    bound = 2 * R.half_step(BF) * ref.abs() + 1e-4 * ref.abs().max()
    y = y.reshape(reps, n, cols)
    for i in range(0, reps, 1025):
        R.check(f"rows from {i * n}", y[i], ref, bound)
    assert (y == y[0]).all()


def test_product_of_many_columns():
    """Rows too long for offsets of 31 bits inside a large tile."""
    check_product(257, 32, (1 << 21) + 8, "none", BF, residual=False)


@pytest.mark.parametrize("rows", [2, 40])
def test_product_of_many_weights(rows):
    E, K, cols = 131, 4096, 16384
    announce(f"mx4 experts {E} of {K} x {cols}, {rows} rows each")
    g = gen(3)
    wq, ws = blocks(cols, K)
    wq.random_(0, 256, generator=g)
    ws.random_(120, 130, generator=g)
    x = [b.random_(0, 256, generator=g) if i == 0 else b.random_(120, 130, generator=g) for i, b in enumerate(blocks(rows, K))]
    far = blocks(E * rows, K)
    far[0] = again(x[0], E)
    for i in range(x[1].shape[0]):
        far[1][i, : E * rows] = again(x[1][i, :rows], E)
    w = [wq.expand(E, *wq.shape).contiguous(), ws.expand(E, *ws.shape).contiguous()]
    assert w[0].numel() > 1 << 32
    y = torch.empty(E * rows, cols, dtype=BF, device=DEV)
    gm.mx4_linear_fwd(gm.make_linear_desc(E * rows, K, cols, dtype=BF, experts=E), *far, *w, y, offsets=offsets_of([rows] * E))
    assert torch.isfinite(y).all() and y.any() and is_again(y, y[:rows])


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm(kind):
    reps, n, d = 17000, 61, 2072
    M = reps * n
    announce(f"norm {kind} {M} x {d}")
    g = gen(4)
    bx, br, bdy, w, b = (normal(g, *s, dtype=BF) for s in ((n, d), (n, d), (n, d), (d,), (d,)))
    small = {k: torch.empty(n, d, dtype=BF, device=DEV) for k in ("y", "h", "dx")}
    stats = [torch.empty(n, device=DEV) if kind == "layer" else None, torch.empty(n, device=DEV)]
    gm.norm_fwd(bx, small["y"], weight=w, bias=b, residual=br, h=small["h"], mean=stats[0], rstd=stats[1], kind=kind)
    gm.norm_bwd(bdy, small["h"], stats[1], small["dx"], mean=stats[0], weight=w, dresidual=bx, kind=kind)
    x, h, y = again(bx, reps), again(br, reps), torch.empty(M, d, dtype=BF, device=DEV)
    assert x.numel() > 1 << 31
    mean, rstd = torch.empty(M, device=DEV) if kind == "layer" else None, torch.empty(M, device=DEV)
    gm.norm_fwd(x, y, weight=w, bias=b, residual=h, h=h, mean=mean, rstd=rstd, kind=kind)
    assert is_again(y, small["y"]) and is_again(h, small["h"])
    dy = again(bdy, reps)
    dw, db = torch.empty(d, dtype=torch.float32, device=DEV).zero_(), torch.empty(d, dtype=torch.float32, device=DEV).zero_()
    gm.norm_bwd(dy, h, rstd, x, mean=mean, weight=w, dresidual=x, dweight=dw, dbias=db, kind=kind, grad_accum=True)
    assert is_again(x, small["dx"])
    m = stats[0] if kind == "layer" else None
    _, rw, rb, _, ew, eb = N.norm_bwd(bdy, small["h"], m, stats[1], w, bx, kind)
    deep = M // 64 + 100   # as norm_reference, of all the rows
    nn = (small["h"].double() - (m.double()[:, None] if m is not None else 0)) * stats[1].double()[:, None]
    R.check("dw", dw, reps * rw, reps * ew + (deep + 2) * R.U32 * reps * (bdy.double() * nn).abs().sum(0))
    R.check("db", db, reps * rb, deep * R.U32 * reps * bdy.double().abs().sum(0))


def test_balance():
    reps, n, E, k = 65700, 256, 136, 2
    T = reps * n
    announce(f"balance {T} x {E}")
    g = gen(5)
    logits = normal(g, n, E, dtype=BF)
    ids, wt = torch.empty(n, k, dtype=torch.int32, device=DEV), torch.empty(n, k, device=DEV)
    gm.moe_route(logits, ids, wt)
    mask = torch.arange(n, device=DEV) % 5 > 0
    far = again(logits, reps)
    assert far.numel() > 1 << 31
    fid, fmask = again(ids, reps), again(mask, reps)
    out = [(torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV), torch.empty(1, device=DEV)) for _ in range(2)]
    gm.moe_balance(logits, ids, *out[0], mask=mask)
    gm.moe_balance(far, fid, *out[1], mask=fmask)
    assert torch.equal(out[1][0], out[0][0] * reps)
    counts, shares, loss = N.balance(logits, ids, mask, "softmax")
    # the order's depth: tokens of a group of lanes (128 workgroups of 64), then lanes, waves and workgroups
    deep = T // (128 * 64) + 200
    R.check("shares", out[1][1], shares, deep * R.U32 * shares + 1e-5 * shares)
    R.check("loss", out[1][2], loss[None], (deep * R.U32 + 1e-5) * loss[None])
    d = torch.empty_like(far)
    gm.moe_balance_bwd(far, fid, out[1][0], d, mask=fmask, dloss=torch.full((1,), float(T), device=DEV))
    assert d.any() and is_again(d, d[:n])
    ref, size = N.balance_bwd(logits, out[0][0], k, mask, float(n), "softmax")
    R.check("dlogits", d[:n], ref, R.half_step(BF) * ref.abs() + 1e-5 * size + R.floor_of(BF))


@pytest.mark.parametrize("M,K,N", [(3, (1 << 24) + 32, 40), (70, (1 << 24) + 96, 72), (300, (1 << 22) + 64, 264)])
def test_product_of_long_rows(M, K, N):
    """Rows nearly as long as they may be, of -1, 0 and 1 under scales of 1: every sum is a whole number below 2^24, so exact."""
    announce(f"mx4 product {M} x {K} x {N}")
    g = gen(6)
    value = torch.tensor([0.0, 1.0, -1.0], device=DEV, dtype=torch.float64)
    code = torch.tensor([0, 2, 10], device=DEV, dtype=U8)

    def operand(rows):
        pick = torch.randint(0, 3, (rows, K), device=DEV, generator=g, dtype=U8).int()
        b = blocks(rows, K)
        b[0].copy_(code[pick[:, ::2]] | code[pick[:, 1::2]] << 4)
        b[1].zero_()
        scales = torch.zeros(b[1].shape[0] * 8, dtype=U8, device=DEV)
        scales[: K // 32] = 127
        b[1][:, :rows] = scales.reshape(-1, 1, 8)
        return b, value[pick]

    (x, xv), (w, wv) = operand(M), operand(N)
    y = torch.empty(M, N, device=DEV)
    gm.mx4_linear_fwd(gm.make_linear_desc(M, K, N, dtype=torch.float32), *x, *w, y)
    assert torch.equal(y.double(), xv @ wv.T)
