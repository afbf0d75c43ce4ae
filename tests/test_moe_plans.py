"""Which kernels the planner takes for the sizes of moe_paths.py: what those sizes are there to test stays what they test.
The planner (host code) is compiled alone and asked on the CPU."""
import glob
import os
import subprocess

import pytest

from gated_mlp_gemms_amd import build as B
from gated_mlp_gemms_amd._lib import LINEAR_ACT_NONE
import gated_mlp_gemms_amd as gm
import moe_paths as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ACTS = {"none": LINEAR_ACT_NONE, **gm._ACTS}


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    """Asks plan_check: lines of input to its lines of output."""
    if not os.path.exists(B.HIPCC):
        pytest.skip("the ROCm compilers are not installed")
    if not glob.glob(os.path.join(B.BUILD, "*.o")):
        B.build()
    tmp = tmp_path_factory.mktemp("plan")
    obj, exe = str(tmp / "plan_check.o"), str(tmp / "plan_check")
    src = os.path.join(ROOT, "tests", "abi_check", "plan_check.cpp")
    for cmd in ([B.HIPCC, "-x", "hip", f"--offload-arch={B.ARCH}", "--cuda-host-only", "-O1", "-std=c++17",
                 "-I", os.path.join(ROOT, "include"), "-I", B.CSRC, "-c", src, "-o", obj],
                [B.HIPCC, "-o", exe, obj,
                 *[o for o in glob.glob(os.path.join(B.BUILD, "*.o")) if os.path.basename(o) != "moe_api.o"]]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr

    def ask(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        out = r.stdout.splitlines()
        assert len(out) == len(lines)
        return out

    return ask


def line(p, phase, which="1 1"):
    return f"{phase} {p.M} {p.K} {p.N} {ACTS[p.act]} {gm._DTYPES[p.dtype]} {len(p.counts or ())} {which}"


def test_plans_are_the_ones_that_the_sizes_stand_for(planner):
    lines, want = [], []
    for p in P.PATHS:
        lines += [line(p, "fwd"), line(p, "bwd")]
        want += [p.fwd, p.bwd]
        if p.counts is None:
            lines += [line(p, "bwd", "1 0"), line(p, "bwd", "0 1")]
            want += [p.alone] * 2
    assert list(zip(lines, planner(lines))) == list(zip(lines, want))


def words(plan):
    return dict(w.split("=") for w in plan.split())


def kernels(p):
    """What a size's forward and backward run, by kind."""
    lay, kind = "experts" if p.counts else "linear", "f32" if p.dtype == "f32" else "16"
    act = "gated" if p.act in gm.GATED_ACTS else "plain"
    part = lambda n: "whole" if int(n) == 1 else "parts"   # noqa: E731
    f = words(p.fwd)
    got = {(lay, kind, act, "fwd", f["tile"], part(f.get("splits", 1)))}
    for b in filter(None, (p.bwd, p.alone)):
        b = words(b)
        if b["form"] == "apart":
            got |= {(lay, kind, "dx", b["dx"], part(b["dx_splits"])), (lay, kind, "dw", b["dw"], part(b["dw_splits"]))}
        elif b["form"] == "group":
            got.add((lay, kind, "group"))
        else:
            got.add((b["form"], kind, b["tile"], part(b["splits"]), "pieces" if int(b["pieces"]) else "experts"))
    return got


def test_sizes_take_every_large_tile():
    """(Streaming, strips and 64 x 64 tiles are what most of test_gpu_moe.py's sizes take.)"""
    w8 = ("256x256w8", "128x128")
    want = {("experts", "16", a, "fwd", t, "whole") for a in ("plain", "gated") for t in w8}
    want |= {("experts", "f32", "plain", "fwd", "128x128", "whole")}
    want |= {("linear", "16", a, "fwd", t, s) for a in ("plain", "gated") for t in ("256x128w8", "128x128") for s in ("whole", "parts")}
    want |= {("linear", "16", a, "fwd", "256x256w8", "whole") for a in ("plain", "gated")}
    want |= {("linear", "16", "plain", "fwd", "256x256w8", "parts")}
    want |= {("linear", "f32", "plain", "fwd", "128x128", s) for s in ("whole", "parts")}
    want |= {("linear", "f32", "gated", "fwd", "128x128", "parts")}
    want |= {("linear", "f32", p, "128x128", s) for p in ("dx", "dw") for s in ("whole", "parts")}
    want |= {("linear", "16", "dw", t, s) for t in (*w8, "256x128w8") for s in ("whole", "parts")}
    want |= {("linear", "16", "dx", t, s) for t in (*w8, "256x128w8") for s in ("whole", "parts")} - {("linear", "16", "dx", "128x128", "whole")}
    want |= {("linear", "16", "group")}
    want |= {("experts", "f32", "128x128", s, "pieces") for s in ("whole", "parts")}
    want |= {("experts", "16", t, s, c) for t in w8 for s in ("whole", "parts") for c in ("pieces", "experts")}
    got = set().union(*(kernels(p) for p in P.PATHS))
    assert not want - got, sorted(want - got)


def test_experts_forwards_that_end_in_halves():
    """The 256 x 256 forwards with more tiles than CUs and a last round of at most half of them."""
    halves = 0
    for p in P.PATHS:
        if p.counts and p.fwd.endswith("256x256w8"):
            units = 128 if p.act in gm.GATED_ACTS else 256
            rows = sum(-(-n // 256) for n in (*p.counts, p.M - sum(p.counts)))
            tiles = rows * -(-p.N // units)
            halves += tiles > 256 and 0 < tiles % 256 <= 128
    assert halves >= 5
