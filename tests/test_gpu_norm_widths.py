"""GPU tests of the norm at widths around the limits of its kernels and of its workgroups' number, with more rows than
workgroups, by test_gpu_norm's checks against float64."""
import pytest

from gpu_helpers import announce
import moe_reference as R
from test_gpu_moe import gen, normal
from test_gpu_norm import F32, check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [300, 1100])
@pytest.mark.parametrize("pieces", [511, 640, 768, 769, 1019, 1020])
@pytest.mark.parametrize("dt", list(R.DT.values()))
def test_column_sums_of_every_number_of_workgroups(M, pieces, dt):
    d = pieces * (4 if dt == F32 else 8)
    kind = "rms" if pieces % 2 else "layer"
    announce(f"norm {M} x {d} {kind} {dt}")
    g = gen(pieces)
    x, r, w, b = make(g, M, d, dt, True)
    h, mean, rstd = check_fwd(x, r, w, b if kind == "layer" else None, kind)
    check_bwd(normal(g, M, d, dtype=dt), h, mean, rstd, w, normal(g, M, d, dtype=dt), kind, True)


@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("pieces", [2047, 2048, 2049, 3001, 8191])
@pytest.mark.parametrize("dt", list(R.DT.values()))
def test_forward_of_wide_rows(M, pieces, dt):
    d = pieces * (4 if dt == F32 else 8)
    for kind in ("layer", "rms"):
        announce(f"norm forward {M} x {d} {kind} {dt}")
        for wide in ((True,) if dt == F32 else (False, True)):
            x, r, w, b = make(gen(pieces + M), M, d, dt, wide)
            check_fwd(x, r, w, b if kind == "layer" else None, kind)
            check_fwd(x, None, None, None, kind)
