"""GPU tests of rows beyond the workgroups that a launch has, so that a workgroup takes several: a small problem's rows repeated,
every repetition of which has to be the small problem's result. What a workgroup keeps between rows (its sums' slots in LDS, their
barriers) matters only there."""
import pytest
import torch

import gated_mlp_gemms_amd as gm
from gpu_helpers import announce
from test_gpu_moe import DEV, gen, normal
from test_gpu_norm import check_bwd, check_fwd

pytestmark = pytest.mark.gpu
U8 = torch.uint8


def again(base, rows):
    """`rows` rows, base's over and over."""
    out = torch.empty(rows, *base.shape[1:], dtype=base.dtype, device=DEV)
    n = base.shape[0]
    whole = rows // n * n
    out[:whole].view(-1, *base.shape).copy_(base.expand(whole // n, *base.shape))
    out[whole:] = base[: rows - whole]
    return out


def assert_again(name, t, base):
    n = base.shape[0]
    whole, step = t.shape[0] // n * n, max(1, (1 << 30) // base.numel()) * n
    for i in range(0, whole, step):
        part = t[i: min(i + step, whole)].view(-1, *base.shape)
        assert (part == base).all(), f"{name}: rows from {i}"
    assert torch.equal(t[whole:], base[: t.shape[0] - whole]), name


# 16-byte pieces a row, rows a workgroup, log2 of a launch's workgroups, type: every width that sums over several waves of a workgroup
BF, F32 = torch.bfloat16, torch.float32
FORWARD = [(65, 2, 20, BF), (193, 1, 20, BF), (257, 2, 20, BF), (385, 1, 20, BF), (2049, 1, 20, F32), (2049, 1, 16, BF),
           (8193, 1, 16, F32)]


@pytest.mark.parametrize("pieces,per,groups,dt", FORWARD)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_forward(pieces, per, groups, dt, kind):
    rows, d = (per * (9 if groups == 16 else 5) << groups) // 4 + 37, pieces * (4 if dt == F32 else 8)
    announce(f"norm forward of {rows} x {d} {dt}, {kind}")
    g = gen(pieces)
    x, r, w = normal(g, 61, d, dtype=dt), normal(g, 61, d, dtype=dt), normal(g, d, dtype=dt)
    x *= torch.linspace(0.25, 4, 61, device=DEV)[:, None].to(dt)   # rows whose sums are far from one another's
    check_fwd(x, None, w, None, kind)
    for residual in (None, r):
        small = dict(y=torch.empty_like(x), rstd=torch.empty(61, device=DEV))
        stats = ["rstd"]
        if kind == "layer":
            small["mean"] = torch.empty(61, device=DEV)
            stats.append("mean")
        h = torch.empty_like(x) if residual is not None else None
        gm.norm_fwd(x, small["y"], weight=w, residual=residual, h=h, kind=kind, **{n: small[n] for n in stats})
        far, y = again(x, rows), torch.empty(rows, d, dtype=dt, device=DEV)
        out = {n: torch.empty(rows, device=DEV) for n in stats}
        fres = again(residual, rows) if residual is not None else None
        gm.norm_fwd(far, y, weight=w, residual=fres, h=far if residual is not None else None, kind=kind, **out)   # (the sum in x's place)
        assert_again("y", y, small["y"])
        if residual is not None:
            assert_again("h", far, h)
        for n in stats:
            assert_again(n, out[n], small[n])
        del far, y, fres


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward_of_long_rows(kind):
    rows, d, dt = (5 << 18) + 37, 2049 * 8, torch.bfloat16
    announce(f"norm backward of {rows} x {d}, {kind}")
    g = gen(9)
    h, w = normal(g, 61, d, dtype=dt) * torch.linspace(0.25, 4, 61, device=DEV)[:, None].to(dt), normal(g, d, dtype=dt)
    _, mean, rstd = check_fwd(h, None, w, None, kind)
    small = torch.empty_like(h)
    check_bwd(h, h, mean, rstd, w, h, kind, False)
    gm.norm_bwd(h, h, rstd, small, mean=mean, weight=w, dresidual=h, kind=kind)   # (one tensor for three: 43 GB each)
    far, dx = again(h, rows), torch.empty(rows, d, dtype=dt, device=DEV)
    gm.norm_bwd(far, far, again(rstd, rows), dx, mean=again(mean, rows) if kind == "layer" else None, weight=w, dresidual=far,
                kind=kind)
    assert_again("dx", dx, small)


# type, columns, rows of the 2^20 workgroups of four waves: 8 rows a wave of 256 values (fp32: 4), so one or two units a row
BLOCKS = [(torch.bfloat16, 32, 1 << 25), (torch.float16, 288, 1 << 24), (torch.float32, 32, 1 << 24)]


@pytest.mark.parametrize("dt,K,most", BLOCKS)
def test_blocks_and_their_values(dt, K, most):
    rows, n = most + most // 8 + 13, 61
    announce(f"mx4 blocks of {rows} x {K} {dt}")

    def blocks(rows):
        return [torch.full(s, 0xEE, dtype=U8, device=DEV) for s in gm.mx4_shapes(rows, K)]

    x = normal(gen(K), n, K, dtype=dt) * torch.linspace(0.01, 9, n, device=DEV)[:, None].to(dt)
    few, many = blocks(n), blocks(rows)
    gm.mx4_quantize(x, *few)
    far = again(x, rows)
    gm.mx4_quantize(far, *many)
    assert_again("codes", many[0], few[0])
    for plane in range(few[1].shape[0]):
        assert_again(f"scales {plane}", many[1][plane, :rows], few[1][plane, :n])
    small = torch.empty_like(x)
    gm.mx4_dequantize(*few, small)
    far.fill_(float("nan"))
    gm.mx4_dequantize(*many, far)
    assert_again("values", far, small)
