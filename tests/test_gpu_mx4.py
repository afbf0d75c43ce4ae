"""GPU tests of microscaled 4-bit floating point against float64: codes and scales have to be equal, products within
bounds that count roundings (moe_reference)."""
import math

import pytest
import torch

import gated_mlp_gemms_amd as gm
import moe_reference as R
import mx4_reference as X
from gpu_helpers import announce
from test_gpu_moe import DEV, gen, normal, offsets_of, poison

pytestmark = pytest.mark.gpu
U8 = torch.uint8


def blocks(rows, K, batch=None):
    return [torch.full(s, 0xEE, dtype=U8, device=DEV) for s in gm.mx4_shapes(rows, K, batch)]


def check_blocks(name, codes, scales, x):
    """Codes, scales and the zeros behind a row's last block."""
    code, scale = X.unpack(codes, scales)
    rc, rs = X.encode(x)
    n = rs.shape[-1]
    assert torch.equal(scale[..., :n], rs), f"{name}: scales"
    assert not scale[..., n:].any(), f"{name}: scales behind the last block"
    bad = (rs == 255).repeat_interleave(32, dim=-1)          # a NaN block's codes do not matter
    assert torch.equal(torch.where(bad, 0, code), torch.where(bad, 0, rc)), f"{name}: codes"


def quantize(x, rows=True, columns=True):
    r, c = x.shape[-2:]
    batch = x.shape[0] if x.dim() == 3 else None
    a = blocks(r, c, batch) if rows else (None, None)
    t = blocks(c, (r + 31) // 32 * 32, batch) if columns else (None, None)
    gm.mx4_quantize(x, a[0], a[1], codes_t=t[0], scales_t=t[1])
    return a, t


SIZES = [  # rows, columns
    (1, 32), (3, 64), (5, 96), (31, 160), (32, 256), (33, 288), (64, 512), (65, 1056), (257, 544), (300, 2080), (9, 8224),
    (1030, 64),
]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", list(R.DT))
def test_quantize(rows, cols, dtype):
    announce(f"mx4 quantize {rows} x {cols} {dtype}")
    g, dt = gen(rows * 10000 + cols), R.DT[dtype]
    x = normal(g, rows, cols, dtype=dt) * torch.exp2(torch.randint(-12, 12, (rows, cols), device=DEV, generator=g)).to(dt)
    a, t = quantize(x)
    check_blocks("rows", *a, x)
    check_blocks("columns", *t, X.transposed(x))
    for only in (True, False):   # one of the two alone
        b = quantize(x, rows=only, columns=not only)[0 if only else 1]
        assert all(torch.equal(p, q) for p, q in zip(b, a if only else t)) or not only
        if not only:
            check_blocks("columns alone", *b, X.transposed(x))
    for (codes, scales), ref in ((a, x), (t, X.transposed(x))):
        for out in R.DT.values():
            v = poison(*ref.shape, dtype=out)
            gm.mx4_dequantize(codes, scales, v)
            assert torch.equal(v, X.rounded(ref).to(out))


def test_quantize_a_batch():
    for dt in R.DT.values():
        x = normal(gen(5), 3, 70, 96, dtype=dt)
        a, t = quantize(x)
        check_blocks("rows", *a, x)
        check_blocks("columns", *t, X.transposed(x))
        v = poison(3, 70, 96, dtype=dt)
        gm.mx4_dequantize(*a, v)
        assert torch.equal(v, X.rounded(x).to(dt))


def test_quantize_odd_columns_transposed():
    """The transposed blocks need no whole blocks of columns."""
    for dt, cols in ((torch.bfloat16, 40), (torch.float16, 8), (torch.float32, 36), (torch.float32, 4)):
        for rows in (1, 31, 100):
            x = normal(gen(cols + rows), rows, cols, dtype=dt)
            _, t = quantize(x, rows=False)
            check_blocks("columns", *t, X.transposed(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_value(dtype):
    """Every 16-bit value, below a largest value of the block of each exponent."""
    dt = R.DT[dtype]
    every = torch.arange(-32768, 32768, device=DEV).to(torch.int16).view(dt)
    every = every[torch.isfinite(every)]
    every = every[: every.numel() // 31 * 31].reshape(-1, 31)
    tops = torch.exp2(torch.arange(-24, 16, device=DEV).double() if dtype == "f16" else torch.arange(-133, 128, 3, device=DEV).double()).to(dt)
    for top in tops:
        x = torch.cat([torch.where(every.abs() > top, top, every), top.expand(every.shape[0], 1)], dim=1)
        a, _ = quantize(x.contiguous(), columns=False)
        check_blocks(f"top {float(top)}", *a, x)


def test_quantize_extremes():
    """Blocks of zeros (either sign), subnormals, the largest values, values at and beside every border; a NaN or an
    infinity makes its own block NaN and no other."""
    for dt in R.DT.values():
        announce(f"mx4 extremes {dt}")
        f = torch.finfo(dt)
        x = torch.zeros(64, 96, dtype=dt, device=DEV)
        x[1] = -0.0
        x[2] = f.smallest_normal
        x[3] = f.smallest_normal * f.eps            # the smallest subnormal
        x[4, ::3] = f.max
        x[5] = -f.max
        x[6, 5] = math.nan
        x[7, 40] = math.inf
        x[8, 95] = -math.inf
        edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], dtype=dt, device=DEV)
        near = torch.cat([edge, edge * (1 + f.eps), edge * (1 - f.eps)])
        x[9, :27], x[9, 31] = near, 4.0
        x[10, :27], x[10, 31] = -near * 2, 8.0
        x[11, :27], x[11, 31] = near.to(dt) * f.smallest_normal, f.smallest_normal * 4
        a, t = quantize(x)
        check_blocks("rows", *a, x)
        check_blocks("columns", *t, X.transposed(x))
        v = poison(64, 96, dtype=dt)
        gm.mx4_dequantize(*a, v)
        ref = X.rounded(x)
        assert torch.equal(torch.isnan(v), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(v.double()), torch.nan_to_num(ref.to(dt).double()))


def test_dequantize_every_code_and_scale():
    """16 codes at 256 scales, in every type (beyond its range infinities, as its cast gives)."""
    code = torch.arange(32, device=DEV).remainder(16).expand(256, 32).contiguous()
    scale = torch.arange(256, device=DEV)[:, None]
    for dt in R.DT.values():
        v = poison(256, 32, dtype=dt)
        gm.mx4_dequantize(*X.pack(code, scale), v)
        ref = X.decode(code, scale).to(dt)
        assert torch.equal(torch.isnan(v), torch.isnan(ref))
        keep = ~torch.isnan(ref)
        assert torch.equal(v[keep], ref[keep])


# ---- products ---------------------------------------------------------------------------------------

def make(g, M, K, N, act, dt, experts, bias, residual, wide=3):
    lead = (experts,) if experts else ()
    gated = act in R.GATED

    def four(*shape, scale):   # any codes, block scales spread over 2 wide + 1 exponents
        code = torch.randint(0, 16, shape, device=DEV, generator=g)
        e = torch.randint(-wide, wide + 1, (*shape[:-1], shape[-1] // 32), device=DEV, generator=g) + round(math.log2(scale / 3)) + 127
        return X.pack(code, e), X.decode(code, e)

    t = {}
    (t["x"], t["xs"]), t["xv"] = four(M, K, scale=1.0)
    (t["w"], t["ws"]), t["wv"] = four(*lead, N, K, scale=K ** -0.5 / 2 ** wide)
    (t["u"], t["us"]), t["uv"] = four(*lead, N, K, scale=K ** -0.5 / 2 ** wide) if gated else ((None, None), None)
    t["bias"] = normal(g, *lead, N, scale=0.3, dtype=dt) if bias else None
    t["bias_up"] = normal(g, *lead, N, scale=0.3, dtype=dt) if bias and gated else None
    t["residual"] = normal(g, M, N, dtype=dt) if residual else None
    return t


def product(desc, t, y, **more):
    gm.mx4_linear_fwd(desc, t["x"], t["xs"], t["w"], t["ws"], y, w_up=t["u"], w_up_scales=t["us"], bias=t["bias"],
                      bias_up=t["bias_up"], **more)


def check_product(M, K, N, act, dt, experts=0, offsets=None, bias=True, residual=True, seed=0):
    announce(f"mx4 M={M} K={K} N={N} {act} {dt} experts={experts} bias={bias} residual={residual}")
    t = make(gen(M * 7 + K * 3 + N + seed), M, K, N, act, dt, experts, bias, residual)
    desc = gm.make_linear_desc(M, K, N, act=act, dtype=dt, experts=experts)
    y, pre = poison(M, N, dtype=dt), poison(M, 2 * N if act in R.GATED else N, dtype=dt)
    product(desc, t, y, residual=t["residual"], offsets=offsets, preact=pre)
    ry, rp, mag = R.linear(act, t["xv"], t["wv"], t["uv"], t["bias"], t["bias_up"], t["residual"], offsets)
    R.check("y", y, ry, R.linear_bound(act, dt, K, ry, rp, mag, N))
    R.check("preact", pre, rp, R.half_step(dt) * rp.abs() + R.sum_err(K, mag) + R.floor_of(dt))
    y2 = t["residual"].clone() if residual else poison(M, N, dtype=dt)
    # in place, without preact: another kernel may do it, whose fp32 steps contract otherwise, within the same bound
    product(desc, t, y2, residual=y2 if residual else None, offsets=offsets)
    R.check("y in place", y2, ry, R.linear_bound(act, dt, K, ry, rp, mag, N))


PRODUCTS = [  # M, K, N
    (1, 32, 8), (1, 4096, 1000), (2, 256, 24), (7, 288, 264), (16, 2080, 136), (17, 544, 72), (33, 64, 8), (48, 4096, 520),
    (64, 512, 128), (65, 96, 136), (128, 1024, 256), (129, 2336, 392), (300, 160, 520), (513, 1056, 264), (1100, 64, 1096),
    (2, 11008, 16),
]


@pytest.mark.parametrize("M,K,N", PRODUCTS)
@pytest.mark.parametrize("dtype", list(R.DT))
def test_products(M, K, N, dtype):
    for i, act in enumerate(R.ACTS):
        check_product(M, K, N, act, R.DT[dtype], bias=i % 3 != 1, residual=i % 2 == 0, seed=i)


@pytest.mark.parametrize("M,K,N", [(4096, 512, 2056), (2100, 2048, 4096), (260, 8224, 264), (3000, 4128, 1544)])
@pytest.mark.parametrize("dtype", list(R.DT))
def test_large_products(M, K, N, dtype):
    for i, act in enumerate(("none", "swiglu", "gelu_tanh")):
        check_product(M, K, N, act, R.DT[dtype])
        # without a residual and pre-activation a large tile's results leave from registers
        check_product(M, K, N, act, R.DT[dtype], residual=False, bias=i != 1)


@pytest.mark.parametrize("act", R.ACTS)
def test_large_products_activations(act):
    for dt in (torch.bfloat16, torch.float16):
        check_product(2049, 288, 2056, act, dt, residual=False)
        check_product(3001, 96, 1544, act, dt, experts=4, offsets=offsets_of([1000, 0, 1500, 401]), residual=False)


PARTS = [  # long K with few tiles: parts of K, on tiles of 64, 128 and 256
    (40, 8224, 264, R.ACTS), (130, 16416, 136, ("none", "geglu")), (300, 12320, 264, ("relu", "swiglu")),
    (775, 30752, 432, ("swiglu",)), (1772, 37536, 1160, ("swiglu",)),
]


@pytest.mark.parametrize("M,K,N,acts", PARTS)
@pytest.mark.parametrize("dtype", list(R.DT))
def test_products_in_parts(M, K, N, acts, dtype):
    for i, act in enumerate(acts):
        desc = gm.make_linear_desc(M, K, N, act=act, dtype=R.DT[dtype])
        assert gm.mx4_linear_workspace_bytes(desc) >= 2 * M * N * 4
        check_product(M, K, N, act, R.DT[dtype], bias=i % 3 != 1, residual=i % 2 == 0, seed=i)


@pytest.mark.parametrize("counts,tail,K,N", [([2500, 0, 2701], 300, 288, 2312), ([4000, 513], 0, 544, 2056)])
@pytest.mark.parametrize("dtype", list(R.DT))
def test_many_rows_of_experts(counts, tail, K, N, dtype):
    for act in ("none", "swiglu"):
        for residual in (True, False):
            check_product(sum(counts) + tail, K, N, act, R.DT[dtype], experts=len(counts), offsets=offsets_of(counts),
                          residual=residual)


EXPERTS = [  # rows an expert, rows behind them, K, N
    ([1], 0, 32, 8), ([0], 3, 64, 24), ([5], 0, 288, 136), ([0, 1, 0, 2], 0, 2080, 72), ([1, 0, 0, 16, 17, 3], 5, 160, 264),
    ([40, 0, 3], 9, 544, 40), ([130, 7, 0, 64, 129], 0, 288, 392), ([0, 0, 300, 0], 20, 96, 136),
    ([700, 100, 0, 300], 0, 160, 264), ([257, 511, 257], 31, 288, 520), ([2001, 65, 1000], 301, 544, 72),
]


@pytest.mark.parametrize("counts,tail,K,N", EXPERTS)
@pytest.mark.parametrize("dtype", list(R.DT))
def test_experts(counts, tail, K, N, dtype):
    for i, act in enumerate(R.ACTS):
        check_product(sum(counts) + tail, K, N, act, R.DT[dtype], experts=len(counts), offsets=offsets_of(counts),
                      bias=i % 3 != 1, residual=i % 2 == 0, seed=i)


@pytest.mark.parametrize("E", [63, 64, 65, 255, 256, 1024])
def test_many_experts(E):
    g = torch.Generator().manual_seed(E)
    few = [int(c) for c in torch.randint(0, 3, (E,), generator=g)]
    many = [int(c) for c in torch.randint(0, 60, (E,), generator=g)]
    for counts in (few, many) if E <= 256 else (few,):
        check_product(sum(counts) + 7, 96, 40, "swiglu", torch.bfloat16, experts=E, offsets=offsets_of(counts))


def test_offsets_out_of_range_stay_inside():
    """Offsets that are no partition give wrong rows, never a store outside y (its neighbours in memory keep their
    values)."""
    g = gen(8)
    K, N, E = 64, 72, 5
    for off in ([0, 50, 20, 900, -3, 100], [-5, -4, -3, -2, -1, 0], [7, 300, 300, 300, 300, 10 ** 9], [0] * 6):
        offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        for M in (200, 40, 3):
            announce(f"mx4 offsets {off} M={M}")
            t = make(g, M, K, N, "swiglu", torch.bfloat16, E, True, False)
            guard = torch.full((3 * M, N), 7.0, dtype=torch.bfloat16, device=DEV)
            product(gm.make_linear_desc(M, K, N, act="swiglu", dtype=torch.bfloat16, experts=E), t, guard[M:2 * M], offsets=offsets)
            assert (guard[:M] == 7).all() and (guard[2 * M:] == 7).all()


def test_nan_blocks_stay_in_their_rows_and_columns():
    g = gen(9)
    for M, K, N in ((3, 512, 40), (150, 512, 264), (600, 288, 520)):
        for dt in (torch.bfloat16, torch.float32):
            announce(f"mx4 nan {M} {K} {N} {dt}")
            t = make(g, M, K, N, "none", dt, 0, False, False)
            desc = gm.make_linear_desc(M, K, N, dtype=dt)
            ref, y = poison(M, N, dtype=dt), poison(M, N, dtype=dt)
            product(desc, t, ref)
            t["xs"][1, M // 2, 0], t["ws"][0, N - 1, 5] = 255, 255
            product(desc, t, y)
            hit = torch.zeros(M, N, dtype=torch.bool, device=DEV)
            hit[M // 2], hit[:, N - 1] = True, True
            assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], ref[~hit])


def test_scales_over_the_whole_range():
    """Products of tiny by huge blocks: exponents far from 0 that meet again."""
    g = gen(10)
    for M, K, N in ((5, 256, 24), (130, 544, 136)):
        for shift in (-100, 60):
            code = [torch.randint(0, 16, (r, K), device=DEV, generator=g) for r in (M, N)]
            e = [torch.full((r, K // 32), 127 + s, device=DEV) for r, s in ((M, shift), (N, -shift))]
            t = dict(zip(("x", "xs"), X.pack(code[0], e[0])), **dict(zip(("w", "ws"), X.pack(code[1], e[1]))), u=None, us=None,
                     bias=None, bias_up=None)
            y = poison(M, N, dtype=torch.float32)
            product(gm.make_linear_desc(M, K, N, dtype=torch.float32), t, y)
            # multiples of 1/4 below 2^24: exact
            assert torch.equal(y.double(), X.decode(code[0], e[0]) @ X.decode(code[1], e[1]).T)


def test_product_of_no_rows():
    for experts in (0, 3):
        t = make(gen(1), 0, 64, 72, "swiglu", torch.bfloat16, experts, False, False)
        off = torch.zeros(experts + 1, dtype=torch.int32, device=DEV) if experts else None
        desc = gm.make_linear_desc(0, 64, 72, act="swiglu", dtype=torch.bfloat16, experts=experts)
        product(desc, t, torch.empty(0, 72, dtype=torch.bfloat16, device=DEV), offsets=off)


@pytest.mark.parametrize("M,K,N", [(1, 64, 32), (50, 96, 160), (300, 544, 288), (1000, 1056, 320)])
@pytest.mark.parametrize("dtype", list(R.DT))
def test_layer_forward_and_backward(M, K, N, dtype):
    """The documented step: weights' blocks both ways, x's and dy's; y, dx and dW against float64 on the rounded values."""
    announce(f"mx4 layer {M} {K} {N} {dtype}")
    g, dt = gen(M + K + N), R.DT[dtype]
    x, w, dy = normal(g, M, K, dtype=dt), normal(g, N, K, scale=K ** -0.5, dtype=dt), normal(g, M, N, dtype=dt)
    (wq, wt), (xq, xt), (gq, gt) = quantize(w), quantize(x), quantize(dy)
    deep = (M + 31) // 32 * 32
    y, dx, dw = poison(M, N, dtype=dt), poison(M, K, dtype=dt), poison(N, K, dtype=dt)
    gm.mx4_linear_fwd(gm.make_linear_desc(M, K, N, dtype=dt), *xq, *wq, y)
    gm.mx4_linear_fwd(gm.make_linear_desc(M, N, K, dtype=dt), *gq, *wt, dx)
    gm.mx4_linear_fwd(gm.make_linear_desc(N, deep, K, dtype=dt), *gt, *xt, dw)
    for name, got, a, b, n in (("y", y, X.rounded(x), X.rounded(w), K), ("dx", dx, X.rounded(dy), X.rounded(X.transposed(w))[:, :N], N),
                               ("dw", dw, X.rounded(X.transposed(dy)), X.rounded(X.transposed(x)), deep)):
        ref = a @ b.T
        R.check(name, got, ref, R.half_step(dt) * ref.abs() + 2 * R.sum_err(n, a.abs() @ b.abs().T) + R.floor_of(dt))
    acc = normal(g, N, K)    # a weight gradient that is added to
    total = acc.clone()
    gm.mx4_linear_fwd(gm.make_linear_desc(N, deep, K, dtype=torch.float32), *gt, *xt, total, residual=total)
    a, b = X.rounded(X.transposed(dy)), X.rounded(X.transposed(x))
    ref = acc.double() + a @ b.T
    R.check("dw added", total, ref, R.U32 * ref.abs() + 2 * R.sum_err(deep, a.abs() @ b.abs().T))


def test_same_bits_again_on_another_stream_and_in_a_graph():
    g, dt = gen(12), torch.bfloat16
    for M, K, N, E in ((9, 2048, 264, 0), (200, 4096, 264, 0), (700, 544, 1032, 0), (333, 288, 264, 7)):
        x, w = normal(g, M, K, dtype=dt), normal(g, *((E,) if E else ()), N, K, scale=K ** -0.5, dtype=dt)
        (wq, ws), _ = quantize(w, columns=False)
        xq, xs = blocks(M, K)
        offsets = offsets_of([M // 7] * 6 + [M - M // 7 * 6]) if E else None
        desc = gm.make_linear_desc(M, K, N, act="relu", dtype=dt, experts=E)
        work = torch.empty(gm.mx4_linear_workspace_bytes(desc), dtype=U8, device=DEV)
        y = poison(M, N, dtype=dt)

        def step(stream=None, workspace=work):
            gm.mx4_quantize(x, xq, xs, stream=stream)
            gm.mx4_linear_fwd(desc, xq, xs, wq, ws, y, offsets=offsets, workspace=workspace, stream=stream)

        step()
        torch.cuda.synchronize()
        first = y.clone()
        side = torch.cuda.Stream()
        for stream in (None, side, side.cuda_stream):
            for workspace in (work, None):
                y.zero_()
                torch.cuda.synchronize()
                step(stream, workspace)
                torch.cuda.synchronize()
                assert torch.equal(first, y)
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            step()
        for i in range(3):
            x.copy_(normal(gen(i), M, K, dtype=dt))
            graph.replay()
            torch.cuda.synchronize()
            replayed = y.clone()
            step()
            torch.cuda.synchronize()
            assert torch.equal(replayed, y)
