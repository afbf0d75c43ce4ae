"""Which kernels the 4-bit products' planner takes around what a launch can hold. The planner (host code) is compiled alone
and asked on the CPU."""
import glob
import os
import subprocess

import pytest

import gated_mlp_gemms_amd as gm
from gated_mlp_gemms_amd import build as B
from gated_mlp_gemms_amd._lib import LINEAR_ACT_NONE

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = (1 << 24) - 1   # tiles of 256 threads that a launch holds
SWIGLU = gm._ACTS["swiglu"]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """(M, K, N, act, experts) to the planner's words as a dict, None where it refuses."""
    if not os.path.exists(B.HIPCC):
        pytest.skip("the ROCm compilers are not installed")
    if not glob.glob(os.path.join(B.BUILD, "*.o")):
        B.build()
    tmp = tmp_path_factory.mktemp("plan")
    obj, exe = str(tmp / "mx4_plan_check.o"), str(tmp / "mx4_plan_check")
    src = os.path.join(ROOT, "tests", "abi_check", "mx4_plan_check.cpp")
    for cmd in ([B.HIPCC, "-x", "hip", f"--offload-arch={B.ARCH}", "--cuda-host-only", "-O1", "-std=c++17",
                 "-I", os.path.join(ROOT, "include"), "-I", B.CSRC, "-c", src, "-o", obj],
                [B.HIPCC, "-o", exe, obj,
                 *[o for o in glob.glob(os.path.join(B.BUILD, "*.o")) if os.path.basename(o) != "mx4_api.o"]]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr

    def ask(*size):
        r = subprocess.run([exe], input=" ".join(str(v) for v in size) + "\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        line = r.stdout.strip()
        return None if line == "refused" else dict(w.split("=") for w in line.split())

    return ask


def row_tiles(M, E, bm):
    return M // bm + min(M, E) + 1 if E else -(-M // bm)


# few rows an expert whose tiles of 16 x 16 are more than a launch holds, each with the next size that is not streamed, and
# products whose 64 x 64 or 128 x 128 tiles are
@pytest.mark.parametrize("M,K,N,act,E", [(2048, 64, 1 << 20, LINEAR_ACT_NONE, 256), (2049, 64, 1 << 20, LINEAR_ACT_NONE, 256),
                                         (8192, 32, 1 << 19, SWIGLU, 1024), (8192, 32, 1 << 21, LINEAR_ACT_NONE, 1024),
                                         (1 << 29, 32, 256, LINEAR_ACT_NONE, 0), (1 << 27, 32, 512, SWIGLU, 0),
                                         (1 << 29, 32, 64, LINEAR_ACT_NONE, 1024)])
def test_sizes_that_larger_tiles_hold(plan, M, K, N, act, E):
    p = plan(M, K, N, act, E)
    assert p is not None and p["form"] != "stream" and 0 < int(p["tiles"]) <= MOST
    bm, bn = (int(v) for v in p["form"].split("x"))
    assert int(p["tiles"]) == row_tiles(M, E, bm) * -(-N // bn) * int(p["splits"])


@pytest.mark.parametrize("M,K,N,act,E", [(8192, 32, 1 << 22, LINEAR_ACT_NONE, 1024), (8192, 32, 1 << 21, SWIGLU, 1024)])
def test_sizes_that_no_tile_holds(plan, M, K, N, act, E):
    assert row_tiles(M, E, 256) * (N // (256 if act == LINEAR_ACT_NONE else 128)) > MOST
    assert plan(M, K, N, act, E) is None
    d = gm.make_linear_desc(M, K, N, act="none" if act == LINEAR_ACT_NONE else "swiglu", dtype="bf16", experts=E)
    with pytest.raises(gm.MlpError, match="threads"):   # the workspace's size refuses what the product refuses
        gm.mx4_linear_workspace_bytes(d)


def test_sizes_that_are_streamed_as_before(plan):
    for M, K, N, act, E in ((16, 4096, 11008, LINEAR_ACT_NONE, 0), (96, 2048, 1376, SWIGLU, 64), (8, 64, (1 << 25) - 8, LINEAR_ACT_NONE, 1),
                            (2047, 64, 1 << 19, LINEAR_ACT_NONE, 256)):
        p = plan(M, K, N, act, E)
        assert p["form"] == "stream" and int(p["tiles"]) == row_tiles(M, E, 16) * -(-N // 16)
    assert plan(17, 4096, 11008, LINEAR_ACT_NONE, 0)["form"] != "stream"
