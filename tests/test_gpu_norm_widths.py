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
