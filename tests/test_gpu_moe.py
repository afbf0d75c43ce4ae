"""GPU tests of the mixture-of-experts operators against float64, over sizes and masks where they can
go wrong. Bounds count roundings (see moe_reference); whole numbers have to be equal."""
import math

import pytest
import torch

import gated_mlp_gemms_amd as gm
import moe_reference as R
from gpu_helpers import announce

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


def poison(*shape, dtype):
    """An output buffer of values that no result has."""
    return torch.full(shape, -12345, dtype=dtype, device=DEV) if dtype in (torch.int32, torch.uint8) \
        else torch.full(shape, float("nan"), dtype=dtype, device=DEV)


# ---- router -------------------------------------------------------------------------------------

ROUTE = [  # T, E, k
    (1, 1, 1), (1, 4, 4), (3, 7, 2), (24, 64, 4), (65, 16, 16), (17, 17, 8), (130, 60, 3), (40, 128, 8), (33, 129, 6),
    (50, 256, 8), (9, 257, 16), (7, 512, 8), (5, 1000, 8), (4, 1024, 16), (5000, 33, 5),
]


def run_route(x, k, score, renorm):
    T = x.shape[0]
    ids, w = poison(T, k, dtype=torch.int32), poison(T, k, dtype=torch.float32)
    gm.moe_route(x, ids, w, score=score, renorm=renorm)
    return ids, w


def check_route(x, k, score, renorm, g):
    T, E = x.shape
    ids, w = run_route(x, k, score, renorm)
    rid, rw, _ = R.route(x, k, score, renorm)
    assert torch.equal(ids.long(), rid)
    # the probabilities are ratios of a sum of E exponentials, each off by its argument's rounding
    span = torch.nan_to_num(x.double(), neginf=0.0).abs().max().item()
    rel = (E + 32 + 4 * span) * R.U32
    R.check("weights", w, rw, rel * rw + 1e-37)
    dw = normal(g, T, k)
    dl = poison(T, E, dtype=x.dtype)
    gm.moe_route_bwd(x, ids, dw, dl, score=score, renorm=renorm)
    ref = R.route_bwd(x, rid, dw, score, renorm)
    mag = (dw.double().abs() * rw).sum(dim=1, keepdim=True) * (2 if renorm or score == "softmax" else 1) + dw.abs().max()
    R.check("dlogits", dl, ref, R.half_step(x.dtype) * ref.abs() + 2 * rel * mag + R.floor_of(x.dtype))


@pytest.mark.parametrize("T,E,k", ROUTE)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, score, renorm):
    for i, dt in enumerate(R.DT.values()):
        announce(f"route T={T} E={E} k={k} {score} renorm={renorm} {dt}")
        g = gen(T * 1000 + E + i)
        check_route(normal(g, T, E, scale=2.0, dtype=dt), k, score, renorm, g)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_ties_masks_and_extremes(score, renorm):
    for dt in R.DT.values():
        announce(f"route masks {score} {renorm} {dt}")
        g = gen(5)
        x = torch.round(normal(g, 64, 70, scale=1.0)).to(dt)      # many ties, both zeros
        x[1] = 0.0
        x[2, ::2] = -0.0
        x[2, 1::2] = 0.0
        x[3] = -math.inf                                          # no expert left
        x[4, 1:] = -math.inf                                      # one left
        x[5, 5:] = -math.inf                                      # fewer left than chosen
        x[6] = torch.finfo(torch.float16).min                     # a mask of the type's lowest value
        x[7, 3] = 60000.0
        x[8] = -80.0
        check_route(x, 8, score, renorm, g)


def test_route_nan_counts_as_the_largest():
    x = normal(gen(1), 3, 20)
    x[1, 11] = math.nan
    ids, w = run_route(x, 2, "softmax", True)
    assert int(ids[1, 0]) == 11 and torch.isnan(w[1]).all() and torch.isfinite(w[[0, 2]]).all()


def test_route_bwd_ignores_ids_out_of_range():
    x, dw = normal(gen(2), 6, 40), normal(gen(3), 6, 4)
    ids, _ = run_route(x, 4, "sigmoid", False)
    some = ids.clone()
    some[:, 2], some[3, 0] = -1, 40
    dl, ref = poison(6, 40, dtype=x.dtype), poison(6, 40, dtype=x.dtype)
    gm.moe_route_bwd(x, some, dw, dl, score="sigmoid", renorm=False)
    masked = torch.where(some == ids, dw, torch.zeros_like(dw))
    gm.moe_route_bwd(x, ids, masked, ref, score="sigmoid", renorm=False)
    assert torch.equal(dl, ref)


# ---- sort and rows ------------------------------------------------------------------------------

SORT = [  # n, E
    (1, 1), (1, 1024), (5, 3), (63, 2), (64, 64), (65, 5), (192, 64), (1000, 7), (4096, 100), (4097, 63), (5003, 1),
    (20000, 256), (70001, 64), (9000, 1023), (6000, 1024),
]


@pytest.mark.parametrize("n,E", SORT)
@pytest.mark.parametrize("kind", ["even", "skewed", "one", "dropped", "all dropped"])
def test_sort(n, E, kind):
    announce(f"sort n={n} E={E} {kind}")
    g = gen(n + E)
    r = torch.rand(n, device=DEV, generator=g)
    ids = {"even": r * E, "skewed": r ** 4 * E, "one": torch.full_like(r, E - 1), "dropped": r * (E + 3) - 2,
           "all dropped": torch.where(r < 0.5, -1.0, float(E))}[kind].floor().to(torch.int32)
    off, row, slot = (poison(m, dtype=torch.int32) for m in (E + 1, n, n))
    gm.moe_sort(ids, E, off, row, slot)
    key = torch.where((ids < 0) | (ids >= E), torch.full_like(ids, E), ids).long()
    want = torch.sort(key, stable=True)[1]
    assert torch.equal(slot.long(), want)
    assert torch.equal(row.long()[want], torch.arange(n, device=DEV))
    assert torch.equal(off.long(), torch.bincount(key, minlength=E + 1).cumsum(0).roll(1).index_fill_(
        0, torch.tensor([0], device=DEV), 0))


def test_sort_of_nothing():
    off = poison(6, dtype=torch.int32)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    gm.moe_sort(none, 5, off, none, none)
    assert torch.equal(off, torch.zeros_like(off))


ROWS = [  # T, E, k, d
    (1, 1, 1, 8), (1, 8, 8, 2048), (3, 4, 2, 16), (48, 64, 4, 2048), (77, 60, 3, 1032), (130, 16, 6, 264),
    (64, 5, 5, 4104), (33, 300, 16, 72), (1000, 12, 2, 520), (20, 8, 1, 8200),
]


@pytest.mark.parametrize("T,E,k,d", ROWS)
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
def test_rows_there_and_back(T, E, k, d, dropped):
    for dt in R.DT.values():
        announce(f"rows T={T} E={E} k={k} d={d} dropped={dropped} {dt}")
        g = gen(T + d)
        n = T * k
        ids = torch.rand(T, E, device=DEV, generator=g).topk(k, dim=1)[1].to(torch.int32)
        ids[torch.rand(T, k, device=DEV, generator=g) < dropped] = -1
        off, row, slot = (poison(m, dtype=torch.int32) for m in (E + 1, n, n))
        gm.moe_sort(ids, E, off, row, slot)
        kept = int(off[E])
        x, res, dout = (normal(g, T, d, dtype=dt) for _ in range(3))
        ys, dxs = (normal(g, n, d, dtype=dt) for _ in range(2))
        ys[kept:], dxs[kept:] = math.nan, math.inf     # a dropped row's content does not matter
        w = torch.rand(T, k, device=DEV, generator=g)
        u, f = R.half_step(dt), R.floor_of(dt)

        xs = poison(n, d, dtype=dt)
        gm.moe_gather(x, slot, off, xs)
        want = torch.zeros_like(xs)
        want[:kept] = x[slot[:kept].long() // k]
        assert torch.equal(xs, want)

        token, sl = slot[:kept].long() // k, slot[:kept].long()
        terms = w.reshape(-1)[sl].double()[:, None] * ys[:kept].double()
        for residual in (res, None):
            out = poison(T, d, dtype=dt)
            gm.moe_combine(ys, w, row, off, out, residual=residual)
            base = residual.double() if residual is not None else torch.zeros(T, d, dtype=torch.float64, device=DEV)
            ref = base.clone().index_add_(0, token, terms)
            mag = base.abs().index_add_(0, token, terms.abs())
            R.check("out", out, ref, u * ref.abs() + (k + 2) * R.U32 * mag + f)
        dys, dw = poison(n, d, dtype=dt), poison(T, k, dtype=torch.float32)
        gm.moe_combine_bwd(dout, ys, w, row, slot, off, dys, dw)
        rd = torch.zeros(n, d, dtype=torch.float64, device=DEV)
        rd[:kept] = w.reshape(-1)[sl].double()[:, None] * dout.double()[token]
        R.check("dys", dys, rd, (u + 2 * R.U32) * rd.abs() + f)
        prod = ys[:kept].double() * dout.double()[token]
        rw, mw = (torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(2))
        rw[sl], mw[sl] = prod.sum(dim=1), prod.abs().sum(dim=1)
        R.check("dweights", dw.reshape(-1), rw, R.sum_err(d, mw))

        dx = poison(T, d, dtype=dt)
        gm.moe_gather_bwd(dxs, row, off, dx)
        z = torch.zeros(T, d, dtype=torch.float64, device=DEV)
        ref, mag = z.clone().index_add_(0, token, dxs[:kept].double()), z.index_add_(0, token, dxs[:kept].double().abs())
        R.check("dx", dx, ref, u * ref.abs() + k * R.U32 * mag + f)


def test_combine_in_place_equals_out_of_place():
    g = gen(9)
    T, E, k, d, dt = 50, 6, 3, 136, torch.bfloat16
    ids = torch.rand(T, E, device=DEV, generator=g).topk(k, dim=1)[1].to(torch.int32)
    off, row, slot = (poison(m, dtype=torch.int32) for m in (E + 1, T * k, T * k))
    gm.moe_sort(ids, E, off, row, slot)
    ys, res, w = normal(g, T * k, d, dtype=dt), normal(g, T, d, dtype=dt), torch.rand(T, k, device=DEV, generator=g)
    out = poison(T, d, dtype=dt)
    gm.moe_combine(ys, w, row, off, out, residual=res)
    gm.moe_combine(ys, w, row, off, res, residual=res)
    assert torch.equal(out, res)


def test_rows_out_of_range_are_skipped():
    """Entries outside their range name no row: zeros, not an access."""
    g = gen(4)
    T, E, k, d = 16, 4, 2, 64
    n = T * k
    x, ys = normal(g, T, d), normal(g, n, d)
    slot = torch.arange(n, device=DEV, dtype=torch.int32)
    slot[3], slot[7] = -1, n
    off = torch.tensor([0, 8, 16, 24, 10 * n], device=DEV, dtype=torch.int32)
    xs, dys, dw = poison(n, d, dtype=x.dtype), poison(n, d, dtype=x.dtype), torch.zeros(T, k, device=DEV)
    gm.moe_gather(x, slot, off, xs)
    good = (slot >= 0) & (slot < n)
    assert torch.equal(xs[good], x[slot[good].long() // k]) and not xs[~good].any()
    row = torch.arange(n, device=DEV, dtype=torch.int32)
    row[5], row[6] = -7, 2 * n
    out = poison(T, d, dtype=x.dtype)
    gm.moe_combine(ys, torch.ones(T, k, device=DEV), row, off, out)
    keep = torch.ones(n, device=DEV)
    keep[5] = keep[6] = 0
    assert torch.equal(out, (ys * keep[:, None]).reshape(T, k, d)[:, 0] + (ys * keep[:, None]).reshape(T, k, d)[:, 1])
    gm.moe_combine_bwd(x, ys, torch.ones(T, k, device=DEV), row, slot, off, dys, dw)
    assert torch.equal(dys[good], x[slot[good].long() // k]) and not dys[~good].any()


# ---- linear layer and experts -------------------------------------------------------------------

def make_linear(g, M, K, N, act, dt, experts, bias, residual):
    lead = (experts,) if experts else ()
    gated = act in R.GATED
    t = dict(x=normal(g, M, K, dtype=dt), w=normal(g, *lead, N, K, scale=K ** -0.5, dtype=dt))
    t["w_up"] = normal(g, *lead, N, K, scale=K ** -0.5, dtype=dt) if gated else None
    t["bias"] = normal(g, *lead, N, scale=0.3, dtype=dt) if bias else None
    t["bias_up"] = normal(g, *lead, N, scale=0.3, dtype=dt) if bias and gated else None
    t["residual"] = normal(g, M, N, dtype=dt) if residual else None
    return t


def check_linear(M, K, N, act, dt, experts=0, offsets=None, bias=True, residual=True, seed=0):
    announce(f"linear M={M} K={K} N={N} {act} {dt} experts={experts} bias={bias} residual={residual}")
    g = gen(M * 7 + K * 3 + N + seed)
    t = make_linear(g, M, K, N, act, dt, experts, bias, residual)
    gated = act in R.GATED
    P = 2 * N if gated else N
    desc = gm.make_linear_desc(M, K, N, act=act, dtype=dt, experts=experts)
    y, pre = poison(M, N, dtype=dt), poison(M, P, dtype=dt)
    gm.linear_fwd(desc, t["x"], t["w"], y, w_up=t["w_up"], bias=t["bias"], bias_up=t["bias_up"],
                  residual=t["residual"], offsets=offsets, preact=pre)
    ry, rp, mag = R.linear(act, t["x"], t["w"], t["w_up"], t["bias"], t["bias_up"], t["residual"], offsets)
    R.check("y", y, ry, R.linear_bound(act, dt, K, ry, rp, mag, N))
    R.check("preact", pre, rp, R.half_step(dt) * rp.abs() + R.sum_err(K, mag) + R.floor_of(dt))
    y2 = poison(M, N, dtype=dt)
    gm.linear_fwd(desc, t["x"], t["w"], y2, w_up=t["w_up"], bias=t["bias"], bias_up=t["bias_up"],
                  residual=t["residual"], offsets=offsets)
    assert torch.equal(y, y2), "without preact"

    dy = normal(g, M, N, dtype=dt)
    kept = int(offsets[-1]) if offsets is not None else M
    saved = pre if act != "none" else None
    if offsets is not None and kept < M:      # what a row of no expert holds does not matter
        dy[kept:] = math.nan
        t["x"][kept:] = math.inf
    ref = R.linear_bwd(act, dy[:kept], t["x"][:kept], t["w"], t["w_up"],
                       saved[:kept] if saved is not None else None, offsets)
    u, f = R.half_step(dt), R.floor_of(dt)
    # dz is rounded to the type (f32: not), independently per element: the sum of those errors stays
    # within 7 roots of the sum of their squared bounds but for one case in 10^10 (Hoeffding); below the
    # type's smallest normal the step is absolute (floor_of), times the factor dz meets
    uz = 0.0 if act == "none" or dt == torch.float32 else u
    z = saved[:kept].double()[:, :N].abs().max().item() if act != "none" and kept else 0.0
    ea = 0.0 if act == "none" else 16 * R.U32 * (1 + z) ** 3    # f, f' in fp32, over the largest z

    def bound(v, mag, root, factors, n):
        return u * v.abs() + R.sum_err(n, mag) + 7 * uz * root + ea * (mag + root) + f * (factors if uz else 0) + f * n

    for accum in (False, True):
        gt = torch.float32 if accum else dt
        made = [poison(*t["w"].shape, dtype=gt) for _ in range(2)] + [poison(*t["w"].shape[:-1], dtype=gt) for _ in range(2)]
        if accum:
            for m in made:
                m.copy_(normal(g, *m.shape))
        before = [m.clone() for m in made]
        dx = poison(M, K, dtype=dt)
        gm.linear_bwd(desc, dy, t["x"], t["w"], w_up=t["w_up"], preact=saved, offsets=offsets, dx=dx, dw=made[0],
                      dw_up=made[1] if gated else None, dbias=made[2], dbias_up=made[3] if gated else None,
                      grad_accum=accum)
        R.check("dx", dx[:kept], ref["dx"][0], bound(*ref["dx"], P))
        assert not dx[kept:].any()
        for i in range(2 if gated else 1):
            v, mag = ref["dw"][i][:2]
            b, mb = ref["db"][i]
            if accum:
                R.check("dw+", made[i], v + before[i].double(), bound(*ref["dw"][i], M) + 2 * R.U32 * (before[i].double().abs() + mag))
                R.check("db+", made[2 + i], b + before[2 + i].double(),
                        R.sum_err(M, mb) + ea * mb + 2 * R.U32 * (before[2 + i].double().abs() + mb) + f * M)
                if offsets is not None:
                    for e, a, z_ in R.spans(offsets, M):
                        if a == z_:
                            assert torch.equal(made[i][e], before[i][e]) and torch.equal(made[2 + i][e], before[2 + i][e])
            else:
                R.check("dw", made[i], v, bound(*ref["dw"][i], M))
                R.check("db", made[2 + i], b, u * b.abs() + R.sum_err(M, mb) + ea * mb + f * (M + 1))
        if accum:
            continue
        # each gradient asked for alone is the same
        alone = poison(M, K, dtype=dt)
        gm.linear_bwd(desc, dy, t["x"], t["w"], w_up=t["w_up"], preact=saved, offsets=offsets, dx=alone)
        R.check("dx alone", alone[:kept], ref["dx"][0], bound(*ref["dx"], P))
        dw = [poison(*t["w"].shape, dtype=dt) for _ in range(2 if gated else 1)]
        gm.linear_bwd(desc, dy, t["x"], t["w"], w_up=t["w_up"], preact=saved, offsets=offsets, dw=dw[0],
                      dw_up=dw[1] if gated else None)
        for i, m in enumerate(dw):
            R.check("dw alone", m, ref["dw"][i][0], bound(*ref["dw"][i], M))
        db = [poison(*t["w"].shape[:-1], dtype=dt) for _ in dw]
        gm.linear_bwd(desc, dy, t["x"], t["w"], w_up=t["w_up"], preact=saved, offsets=offsets, dbias=db[0],
                      dbias_up=db[1] if gated else None)
        for i, m in enumerate(db):
            assert torch.equal(m, made[2 + i])


LINEAR = [  # M, K, N
    (1, 8, 8), (1, 264, 1000), (2, 4096, 24), (9, 2056, 264), (16, 136, 8200), (17, 72, 264), (64, 520, 136),
    (65, 8, 8), (100, 2048, 128), (129, 264, 392), (300, 136, 520), (513, 1032, 264), (1100, 72, 1096),
]


@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("dtype", list(R.DT))
def test_linear(M, K, N, dtype):
    for i, act in enumerate(R.ACTS):
        check_linear(M, K, N, act, R.DT[dtype], bias=i % 3 != 1, residual=i % 2 == 0, seed=i)


@pytest.mark.parametrize("M,K,N", [(4096, 512, 2056), (2100, 2048, 4096), (260, 8200, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_large(M, K, N, dtype):
    for act in ("none", "gelu_tanh", "swiglu"):
        check_linear(M, K, N, act, R.DT[dtype])


def test_linear_fp32_odd_widths():
    for act in ("none", "geglu"):
        check_linear(70, 260, 516, act, torch.float32)
        check_linear(3, 4, 12, act, torch.float32)


@pytest.mark.parametrize("dtype", list(R.DT))
def test_linear_of_no_rows(dtype):
    dt = R.DT[dtype]
    for experts in (0, 3):
        lead = (experts,) if experts else ()
        desc = gm.make_linear_desc(0, 64, 72, act="swiglu", dtype=dt, experts=experts)
        x, y, pre = (torch.empty(0, m, dtype=dt, device=DEV) for m in (64, 72, 144))
        w, dw, dw_up = (poison(*lead, 72, 64, dtype=dt) for _ in range(3))
        db, db_up = poison(*lead, 72, dtype=dt), poison(*lead, 72, dtype=dt)
        off = torch.zeros(experts + 1, dtype=torch.int32, device=DEV) if experts else None
        gm.linear_fwd(desc, x, w, y, w_up=w, offsets=off, preact=pre)
        gm.linear_bwd(desc, y, x, w, w_up=w, preact=pre, offsets=off, dx=x, dw=dw, dw_up=dw_up, dbias=db, dbias_up=db_up)
        assert not (dw.any() or dw_up.any() or db.any() or db_up.any())


def offsets_of(counts):
    return torch.tensor([0] + counts, device=DEV).cumsum(0).to(torch.int32)


EXPERTS = [  # rows an expert, rows behind them, K, N
    ([1], 0, 8, 8), ([0], 3, 16, 24), ([5], 0, 264, 136), ([0, 1, 0, 2], 0, 2056, 72), ([1, 0, 0, 16, 17, 3], 5, 136, 264),
    ([40, 0, 3], 9, 520, 40), ([130, 7, 0, 64, 129], 0, 264, 392), ([0, 0, 300, 0], 20, 72, 136),
    ([700, 100, 0, 300], 0, 136, 264), ([256, 512, 257], 31, 136, 520), ([2000, 65, 1000], 300, 520, 72),
]


@pytest.mark.parametrize("counts,tail,K,N", EXPERTS)
@pytest.mark.parametrize("dtype", list(R.DT))
def test_experts(counts, tail, K, N, dtype):
    for i, act in enumerate(R.ACTS):
        check_linear(sum(counts) + tail, K, N, act, R.DT[dtype], experts=len(counts), offsets=offsets_of(counts),
                     bias=i % 3 != 1, residual=i % 2 == 0, seed=i)


@pytest.mark.parametrize("E", [63, 64, 65, 200, 1024])
@pytest.mark.parametrize("dtype", list(R.DT))
def test_many_experts(E, dtype):
    g = torch.Generator().manual_seed(E)
    few = [int(c) for c in torch.randint(0, 3, (E,), generator=g)]
    many = [int(c) for c in torch.randint(0, 100, (E,), generator=g)]
    for counts in (few, many) if E <= 200 else (few,):
        check_linear(sum(counts) + 7, 72, 40, "swiglu", R.DT[dtype], experts=E, offsets=offsets_of(counts))


def test_offsets_out_of_range_stay_inside():
    """Offsets that are no partition give wrong rows, never an access outside the tensors (their
    neighbours in memory keep their values)."""
    g = gen(8)
    M, K, N, E = 200, 64, 72, 5
    for off in ([0, 50, 20, 900, -3, 100], [-5, -4, -3, -2, -1, 0], [7, 300, 300, 300, 300, 10 ** 9], [0] * 6):
        offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        for dt in (torch.bfloat16, torch.float32):
            for M_ in (M, 40):
                announce(f"offsets {off} {dt} M={M_}")
                t = make_linear(g, M_, K, N, "swiglu", dt, E, True, False)
                desc = gm.make_linear_desc(M_, K, N, act="swiglu", dtype=dt, experts=E)
                guard = torch.full((3 * M_, N), 7.0, dtype=dt, device=DEV)
                y, pre = guard[M_:2 * M_], torch.zeros(M_, 2 * N, dtype=dt, device=DEV)
                gm.linear_fwd(desc, t["x"], t["w"], y, w_up=t["w_up"], bias=t["bias"], bias_up=t["bias_up"],
                              offsets=offsets, preact=pre)
                wide = torch.full((3 * M_, K), 7.0, dtype=dt, device=DEV)
                wg = torch.full((3 * E, N, K), 7.0, dtype=dt, device=DEV)
                db = torch.full((3 * E, N), 7.0, dtype=dt, device=DEV)
                gm.linear_bwd(desc, torch.zeros(M_, N, dtype=dt, device=DEV), t["x"], t["w"], w_up=t["w_up"], preact=pre,
                              offsets=offsets, dx=wide[M_:2 * M_], dw=wg[E:2 * E], dw_up=torch.empty_like(t["w"]),
                              dbias=db[E:2 * E], dbias_up=torch.empty_like(db[:E]))
                torch.cuda.synchronize()
                for whole, n in ((guard, M_), (wide, M_), (wg, E), (db, E)):
                    assert (whole[:n] == 7.0).all() and (whole[2 * n:] == 7.0).all()


# ---- a whole layer ------------------------------------------------------------------------------

class Layer:
    """A layer of gated experts on a residual stream, forward and backward, on fixed buffers."""

    def __init__(self, T, E, k, d, h, dt, seed=0):
        g = gen(seed)
        n = T * k
        self.x, self.dout = normal(g, T, d, dtype=dt), normal(g, T, d, dtype=dt)
        self.router = normal(g, E, d, scale=d ** -0.5, dtype=dt)
        self.wg, self.wu = normal(g, E, h, d, scale=d ** -0.5, dtype=dt), normal(g, E, h, d, scale=d ** -0.5, dtype=dt)
        self.wd = normal(g, E, d, h, scale=h ** -0.5, dtype=dt)
        new = lambda *s, t=dt: torch.zeros(*s, dtype=t, device=DEV)   # noqa: E731
        i32, f32 = torch.int32, torch.float32
        self.logits, self.ids, self.w = new(T, E), new(T, k, t=i32), new(T, k, t=f32)
        self.off, self.row, self.slot = new(E + 1, t=i32), new(n, t=i32), new(n, t=i32)
        self.xs, self.pre, self.a, self.ys, self.out = new(n, d), new(n, 2 * h), new(n, h), new(n, d), new(T, d)
        self.dys, self.dwt, self.da, self.dxs = new(n, d), new(T, k, t=f32), new(n, h), new(n, d)
        self.dwg, self.dwu, self.dwd = new(E, h, d), new(E, h, d), new(E, d, h)
        self.dlogits, self.dx, self.dxr, self.drouter = new(T, E), new(T, d), new(T, d), new(E, d)
        self.lr = gm.make_linear_desc(T, d, E, dtype=dt)
        self.up = gm.make_linear_desc(n, d, h, act="swiglu", dtype=dt, experts=E)
        self.down = gm.make_linear_desc(n, h, d, dtype=dt, experts=E)
        self.E = E
        byte = lambda b: new(b, t=torch.uint8)   # noqa: E731
        self.ws = {name: byte(gm.linear_workspace_bytes(desc, ph)) for name, desc, ph in (
            ("r", self.lr, "fwd"), ("u", self.up, "fwd"), ("d", self.down, "fwd"), ("rb", self.lr, "bwd"),
            ("ub", self.up, "bwd"), ("db", self.down, "bwd"))}
        self.ws["s"] = byte(gm.moe_sort_workspace_bytes(n, E))

    def step(self):
        s, ws = self, self.ws
        gm.linear_fwd(s.lr, s.x, s.router, s.logits, workspace=ws["r"])
        gm.moe_route(s.logits, s.ids, s.w)
        gm.moe_sort(s.ids, s.E, s.off, s.row, s.slot, workspace=ws["s"])
        gm.moe_gather(s.x, s.slot, s.off, s.xs)
        gm.linear_fwd(s.up, s.xs, s.wg, s.a, w_up=s.wu, offsets=s.off, preact=s.pre, workspace=ws["u"])
        gm.linear_fwd(s.down, s.a, s.wd, s.ys, offsets=s.off, workspace=ws["d"])
        gm.moe_combine(s.ys, s.w, s.row, s.off, s.out, residual=s.x)
        gm.moe_combine_bwd(s.dout, s.ys, s.w, s.row, s.slot, s.off, s.dys, s.dwt)
        gm.linear_bwd(s.down, s.dys, s.a, s.wd, offsets=s.off, dx=s.da, dw=s.dwd, workspace=ws["db"])
        gm.linear_bwd(s.up, s.da, s.xs, s.wg, w_up=s.wu, preact=s.pre, offsets=s.off, dx=s.dxs, dw=s.dwg, dw_up=s.dwu,
                      workspace=ws["ub"])
        gm.moe_gather_bwd(s.dxs, s.row, s.off, s.dx)
        gm.moe_route_bwd(s.logits, s.ids, s.dwt, s.dlogits)
        gm.linear_bwd(s.lr, s.dlogits, s.x, s.router, dx=s.dxr, dw=s.drouter, workspace=ws["rb"])

    def outputs(self):
        return {n: getattr(self, n) for n in ("out", "dx", "dxr", "dwg", "dwu", "dwd", "drouter", "ids", "w", "off")}


def layer_in_double(x, router, wg, wu, wd, ids):
    """The layer's output in float64 with the choice of experts given, differentiable."""
    logits = x @ router.T
    w = torch.softmax(logits.gather(1, ids), dim=1)
    out = x
    for j in range(ids.shape[1]):
        e = ids[:, j]
        g, u = (torch.einsum("td,thd->th", x, m[e]) for m in (wg, wu))
        out = out + w[:, j:j + 1] * torch.einsum("th,tdh->td", torch.nn.functional.silu(g) * u, wd[e])
    return out


def test_layer_gradients_against_double_and_differences():
    """fp32, the whole layer: against autograd of the formula in float64 on the CPU, and against central
    differences of that formula along random directions."""
    L = Layer(37, 8, 2, 32, 40, torch.float32, seed=3)
    L.step()
    leaves = [t.double().cpu().requires_grad_() for t in (L.x, L.router, L.wg, L.wu, L.wd)]
    ids, dout = L.ids.long().cpu(), L.dout.double().cpu()
    out = layer_in_double(*leaves, ids)
    grads = torch.autograd.grad((out * dout).sum(), leaves)
    got = [L.dout + L.dx + L.dxr, L.drouter, L.dwg, L.dwu, L.dwd]
    # five products deep, sums of at most 74 terms of order one: 2000 half steps of the largest value
    for name, a, b in [("out", L.out, out.detach())] + list(zip(("dx", "drouter", "dwg", "dwu", "dwd"), got, grads)):
        R.check(name, a.cpu(), b, torch.full_like(b, 2000 * R.U32 * b.abs().max().item()))
    g = torch.Generator().manual_seed(1)
    h = 1e-5
    with torch.no_grad():
        for leaf, mine in zip(range(5), got):
            v = torch.randn(leaves[leaf].shape, generator=g, dtype=torch.float64)
            moved = [[t + s * h * v if i == leaf else t for i, t in enumerate(leaves)] for s in (1, -1)]
            diff = sum(s * (layer_in_double(*m, ids) * dout).sum() for s, m in zip((1, -1), moved)) / (2 * h)
            along = (mine.double().cpu() * v).sum()
            # the difference is off by h^2 of a third derivative and by double's rounding over h
            scale = (mine.double().cpu().abs() * v.abs()).sum().item()
            assert abs(along.item() - diff.item()) <= 2000 * R.U32 * scale + 1e-6 * scale


@pytest.mark.parametrize("T", [3, 300])
def test_layer_in_a_graph(T):
    """The whole step captured once and replayed with new inputs, an eager step between the replays."""
    L = Layer(T, 8, 2, 128, 264, torch.bfloat16, seed=4)
    L.step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        L.step()
    for i in range(4):
        L.x.copy_(normal(gen(50 + i), *L.x.shape, dtype=torch.bfloat16))
        L.dout.copy_(normal(gen(90 + i), *L.x.shape, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        replayed = {n: t.clone() for n, t in L.outputs().items()}
        L.step()
        torch.cuda.synchronize()
        for n, t in L.outputs().items():
            assert torch.equal(replayed[n], t), (i, n)


def test_layer_on_another_stream_and_twice():
    """The same bits on a stream of the caller's, and on every run."""
    L = Layer(130, 16, 4, 64, 72, torch.bfloat16, seed=6)
    L.step()
    torch.cuda.synchronize()
    first = {n: t.clone() for n, t in L.outputs().items()}
    side = torch.cuda.Stream()
    for t in L.outputs().values():
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.step()
    side.synchronize()
    for n, t in L.outputs().items():
        assert torch.equal(first[n], t), n


@pytest.mark.parametrize("dtype", list(R.DT))
def test_streamed_rows_equal_cached_ones(dtype):
    """From 100 MB of sorted rows on they are streamed: the same values as of the same rows in parts."""
    g, dt = gen(21), R.DT[dtype]
    d = 2048 if dt == torch.float32 else 4096
    T, E, k = 4500, 20, 3
    assert T * k * d * torch.empty(0, dtype=dt).element_size() >= 100 << 20
    n, h = T * k, T // 2
    ids = torch.rand(T, E, device=DEV, generator=g).topk(k, dim=1)[1].to(torch.int32)
    ids[torch.rand(T, k, device=DEV, generator=g) < 0.1] = -1
    off, row, slot = (poison(m, dtype=torch.int32) for m in (E + 1, n, n))
    gm.moe_sort(ids, E, off, row, slot)
    kept = int(off[E])
    x, ys, w = normal(g, T, d, dtype=dt), normal(g, n, d, dtype=dt), torch.rand(T, k, device=DEV, generator=g)
    xs, out, dx, dys, dw = (poison(*s, dtype=t) for s, t in (((n, d), dt), ((T, d), dt), ((T, d), dt), ((n, d), dt),
                                                            ((T, k), torch.float32)))
    gm.moe_gather(x, slot, off, xs)
    assert torch.equal(xs[:kept], x[slot[:kept].long() // k]) and not xs[kept:].any()
    gm.moe_combine(ys, w, row, off, out, residual=x)
    gm.moe_gather_bwd(ys, row, off, dx)
    gm.moe_combine_bwd(x, ys, w, row, slot, off, dys, dw)
    # halves of the tokens, each a smaller problem of its own: every slot of the first expert, in token order
    for a, b in ((0, h), (h, T)):
        m = (b - a) * k
        live = ids[a:b].reshape(-1) >= 0
        part = torch.where(live, 0, -1).to(torch.int32)
        o1, r1, s1 = (poison(c, dtype=torch.int32) for c in (k + 1, m, m))
        gm.moe_sort(part, k, o1, r1, s1)
        ys1 = ys[row[a * k:b * k].long()][s1.long()].contiguous()
        out1, dx1, dys1, dw1 = (poison(*s, dtype=t) for s, t in (((b - a, d), dt), ((b - a, d), dt), ((m, d), dt),
                                                                 ((b - a, k), torch.float32)))
        gm.moe_combine(ys1, w[a:b].contiguous(), r1, o1, out1, residual=x[a:b].contiguous())
        gm.moe_gather_bwd(ys1, r1, o1, dx1)
        gm.moe_combine_bwd(x[a:b].contiguous(), ys1, w[a:b].contiguous(), r1, s1, o1, dys1, dw1)
        assert torch.equal(out[a:b], out1) and torch.equal(dx[a:b], dx1) and torch.equal(dw[a:b], dw1)
        assert torch.equal(dys[row[a * k:b * k].long()][s1.long()], dys1)


@pytest.mark.parametrize("M,K,N,act", [(8192, 2048, 4864, "gelu_tanh"), (4100, 1544, 8200, "none"), (6000, 2056, 2312, "swiglu"),
                                       (9000, 1032, 2056, "reglu"), (3080, 4096, 4096, "relu")])
def test_linear_backward_in_one_launch(M, K, N, act):
    """Sizes whose dx and dW may share a launch, ragged ones among them."""
    for dt in (torch.bfloat16, torch.float16):
        check_linear(M, K, N, act, dt, bias=False, residual=False)


FEW_ROWS = [  # rows an expert, rows behind them, K, N, activations
    ([3, 0, 31, 64, 65, 1, 0, 100], 5, 264, 456, ("none", "swiglu")),          # whole and part K-steps, several tiles a strip
    ([2] * 40 + [0] * 5 + [900], 0, 520, 200, ("gelu_tanh", "glu")),           # one expert summed over pieces
    ([1], 0, 4104, 1288, ("relu", "geglu")), ([7, 12], 0, 1032, 72, ("none", "reglu")),
    ([130, 250, 200, 60], 9, 136, 392, ("relu_sq", "swiglu")),
    ([9, 20, 0, 33], 0, 4096, 4096, ("none",)), ([5, 2, 1, 0], 0, 4104, 4096, ("none",)),   # past the caches, or not in whole lines
    ([200, 90, 140], 0, 4096, 4608, ("none",)),                                # tiles, past the caches
]


@pytest.mark.parametrize("case", FEW_ROWS, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[2]}-{c[3]}")
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_backward_of_few_rows(case, dtype):
    counts, tail, K, N, acts = case
    for act in acts:
        check_linear(sum(counts) + tail, K, N, act, R.DT[dtype], experts=len(counts), offsets=offsets_of(counts))
        if len(counts) <= 2:
            check_linear(sum(counts), K, N, act, R.DT[dtype])


def test_backward_of_few_rows_is_the_same_again():
    dt, g = torch.bfloat16, gen(77)
    for counts, K, N in (([3, 0, 40, 9], 264, 456), ([2] * 40 + [900], 520, 200)):
        M, E = sum(counts), len(counts)
        t = make_linear(g, M, K, N, "none", dt, E, False, False)
        desc, dy, off = gm.make_linear_desc(M, K, N, dtype=dt, experts=E), normal(g, M, N, dtype=dt), offsets_of(counts)
        runs = []
        for _ in range(3):
            dx, dw = poison(M, K, dtype=dt), poison(E, N, K, dtype=dt)
            gm.linear_bwd(desc, dy, t["x"], t["w"], offsets=off, dx=dx, dw=dw)
            runs.append((dx, dw))
        assert all(torch.equal(runs[0][i], r[i]) for r in runs[1:] for i in range(2))


@pytest.mark.parametrize("act,score,bias,experts", [("swiglu", "softmax", False, 8), ("relu_sq", "sigmoid", True, 8),
                                                    ("geglu", "softmax", True, 8), ("swiglu", "sigmoid", True, 7)])
def test_runner_against_double(act, score, bias, experts):
    """The layer's runner, fp32, against autograd of the formula in float64 on the CPU."""
    from gated_mlp_gemms_amd.moe_runner import MoeRunner, moe_tensors

    size = dict(act=act, dtype="f32", tokens=45, width=32, hidden=40, experts=experts)
    t = moe_tensors(seed=5, bias=bias, **size)
    r = MoeRunner(choices=3, score=score, tensors=t, **size)
    r.step()
    infer = MoeRunner(choices=3, score=score, tensors=t, train=False, **size)
    assert torch.equal(infer.forward_infer(), r.out)
    leaf = {k: v.double().cpu().requires_grad_() for k, v in t.items() if k != "dout"}
    gated, ids = act in R.GATED, r.ids.long().cpu()
    x, w1, w2 = leaf["x"], leaf["w_gate" if gated else "w1"], leaf["w_down" if gated else "w2"]
    p = x @ leaf["router"].T
    p = torch.softmax(p, 1) if score == "softmax" else torch.sigmoid(p)
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    out = x
    for j in range(3):
        e = ids[:, j]
        g = (w1[e] @ x[:, :, None])[:, :, 0] + (leaf["b_gate" if gated else "b1"][e] if bias else 0)
        if gated:
            u = (leaf["w_up"][e] @ x[:, :, None])[:, :, 0] + (leaf["b_up"][e] if bias else 0)
            a = (torch.nn.functional.silu(g) if act == "swiglu" else torch.nn.functional.gelu(g, approximate="tanh")) * u
        else:
            a = torch.relu(g) ** 2
        out = out + w[:, j:j + 1] * ((w2[e] @ a[:, :, None])[:, :, 0] + (leaf["b_down" if gated else "b2"][e] if bias else 0))
    names = ["x", "router", "w_gate" if gated else "w1", "w_down" if gated else "w2"] + (["w_up"] if gated else [])
    keys = ["dx", "d_router", "dw1", "dw2"] + (["dw_up"] if gated else [])
    if bias:
        names += ["b_gate" if gated else "b1", "b_down" if gated else "b2"] + (["b_up"] if gated else [])
        keys += ["db1", "db2"] + (["db_up"] if gated else [])
    grads = torch.autograd.grad((out * t["dout"].double().cpu()).sum(), [leaf[n] for n in names])
    # as test_layer_gradients_against_double_and_differences
    R.check("out", r.out.cpu(), out.detach(), torch.full_like(out, 2000 * R.U32 * out.abs().max().item()).detach())
    assert sorted(r.grads()) == sorted(keys)
    for k, b in zip(keys, grads):
        R.check(k, r.grads()[k].cpu(), b, torch.full_like(b, 2000 * R.U32 * b.abs().max().item()))


def test_runner_command(capsys):
    from gated_mlp_gemms_amd import moe_runner

    moe_runner.main(["--tokens", "64", "--width", "64", "--hidden", "72", "--experts", "4", "--choices", "2", "--steps", "2",
                     "--decode-tokens", "3"])
    text = capsys.readouterr().out
    assert "training step, 64 tokens" in text and "in a graph, 3 tokens" in text


def test_calls_on_a_stream_that_is_passed():
    """A torch stream and its handle as the `stream` argument: the same bits as on the current one."""
    g, dt = gen(31), torch.bfloat16
    T, E, k, d = 33, 8, 2, 72
    x, logits = normal(g, T, d, dtype=dt), normal(g, T, E)
    w, b = normal(g, E, d, d, scale=0.1, dtype=dt), normal(g, E, d, dtype=dt)
    desc = gm.make_linear_desc(T * k, d, d, act="relu", dtype=dt, experts=E)
    side = torch.cuda.Stream()

    def run(stream):
        ids, wt = poison(T, k, dtype=torch.int32), poison(T, k, dtype=torch.float32)
        off, row, slot = (poison(n, dtype=torch.int32) for n in (E + 1, T * k, T * k))
        xs, y, out, pre = (poison(n, d, dtype=dt) for n in (T * k, T * k, T, T * k))
        dw, db, dx = poison(E, d, d, dtype=dt), poison(E, d, dtype=dt), poison(T * k, d, dtype=dt)
        ws = [torch.zeros(gm.linear_workspace_bytes(desc, p), dtype=torch.uint8, device=DEV) for p in ("fwd", "bwd")]
        sw = torch.zeros(gm.moe_sort_workspace_bytes(T * k, E), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        gm.moe_route(logits, ids, wt, stream=stream)
        gm.moe_sort(ids, E, off, row, slot, workspace=sw, stream=stream)
        gm.moe_gather(x, slot, off, xs, stream=stream)
        gm.linear_fwd(desc, xs, w, y, bias=b, offsets=off, preact=pre, workspace=ws[0], stream=stream)
        gm.moe_combine(y, wt, row, off, out, residual=x, stream=stream)
        gm.linear_bwd(desc, y, xs, w, preact=pre, offsets=off, dx=dx, dw=dw, dbias=db, workspace=ws[1], stream=stream)
        torch.cuda.synchronize()
        return ids, wt, off, row, slot, xs, y, out, dx, dw, db

    first = run(None)
    for stream in (side, side.cuda_stream):
        assert all(torch.equal(a, c) for a, c in zip(first, run(stream)))
