"""GPU tests of 4-bit products whose 16 x 16 tiles would be more than a launch holds, so that larger tiles take them though their
rows are few."""
import pytest
import torch

import gated_mlp_gemms_amd as gm
from gpu_helpers import announce
from test_gpu_moe import DEV, gen, offsets_of

pytestmark = pytest.mark.gpu
U8, BF = torch.uint8, torch.bfloat16


@pytest.mark.parametrize("act,N", [("none", 1 << 20), ("swiglu", 1 << 20)])
def test_few_rows_an_expert_of_a_very_wide_weight(act, N):
    """256 experts of the same weight and the same 8 rows each: every one has to be what one expert alone gives. Scales are 1 and
    codes' products multiples of 0.25 up to 36, so sums of 64 of them are exact in any order."""
    E, rows, K = 256, 8, 64
    announce(f"mx4 {act} {E} experts of {rows} rows, {K} x {N}")
    gated, g = act == "swiglu", gen(7)

    def operand(n):
        codes, scales = (torch.empty(s, dtype=U8, device=DEV) for s in gm.mx4_shapes(n, K))
        scales.zero_()
        scales[0, :n, : K // 32] = 127
        return codes.random_(0, 256, generator=g), scales

    x, ws = operand(rows), [operand(N) for _ in range(2 if gated else 1)]
    up = lambda w: dict(w_up=w[1][0], w_up_scales=w[1][1]) if gated else {}   # noqa: E731
    one = torch.empty(rows, N, dtype=BF, device=DEV)
    gm.mx4_linear_fwd(gm.make_linear_desc(rows, K, N, act=act, dtype=BF), *x, *ws[0], one, **up(ws))
    assert torch.isfinite(one).all() and one.any()

    M = E * rows
    codes, scales = (torch.empty(s, dtype=U8, device=DEV) for s in gm.mx4_shapes(M, K))
    codes.copy_(x[0].repeat(E, 1))
    scales.zero_()
    scales[:, :M] = x[1][:, :rows].repeat(1, E, 1)
    many = [tuple(t.expand(E, *t.shape).contiguous() for t in w) for w in ws]
    y = torch.full((M, N), float("nan"), dtype=BF, device=DEV)
    gm.mx4_linear_fwd(gm.make_linear_desc(M, K, N, act=act, dtype=BF, experts=E), codes, scales, *many[0], y,
                      offsets=offsets_of([rows] * E), **up(many))
    for e in range(E):
        assert torch.equal(y[e * rows: (e + 1) * rows], one), e
