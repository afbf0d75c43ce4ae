"""CPU tests of the norm's and the balance loss' entry points: every declared symbol is there, arguments are refused on
the host before any HIP call, workspaces are sized, and the float64 references agree with differences of themselves.
No call below reaches a GPU."""
import ctypes as C
import math
import os
import re

import pytest
import torch

import gated_mlp_gemms_amd as gm
import norm_reference as N
from gated_mlp_gemms_amd import _lib
from gated_mlp_gemms_amd._lib import MLP_ERR_ALIGNMENT, MLP_ERR_INVALID_ARG, MLP_ERR_UNSUPPORTED, MLP_ERR_WORKSPACE, MLP_OK

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000      # 16-byte aligned, never dereferenced: each call fails validation first
F32, BF16, F16 = 0, 1, 2
I32 = torch.int32


def err():
    return gm.lib().mlp_last_error().decode()


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "norm.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(norm_\w+)\s*\(", text))
    assert names == set(_lib._NORM_SIGNATURES)
    for n in names:
        assert hasattr(gm.lib(), n) and hasattr(gm, n), n
    assert C.sizeof(_lib.NormDesc) == 32


def desc(M=5, d=64, dtype=BF16, wdtype=BF16, kind=0, eps=1e-5):
    return _lib.NormDesc(M, d, dtype, wdtype, kind, eps)


def fwd(q, x=FAKE, res=None, w=FAKE, b=FAKE, y=FAKE, h=None, mean=FAKE, rstd=FAKE):
    return gm.lib().norm_fwd(C.byref(q) if q else None, x, res, w, b, y, h, mean, rstd, None)


def bwd(q, dy=FAKE, h=FAKE, mean=FAKE, rstd=FAKE, w=FAKE, dres=None, dx=FAKE, dw=FAKE, db=FAKE, acc=0, ws=FAKE, nws=1 << 40):
    return gm.lib().norm_bwd(C.byref(q) if q else None, dy, h, mean, rstd, w, dres, dx, dw, db, acc, ws, nws, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_descriptor_checks(call):
    assert call(None) == MLP_ERR_INVALID_ARG and "desc is NULL" in err()
    assert call(desc(dtype=3)) == MLP_ERR_INVALID_ARG and "dtype" in err()
    assert call(desc(dtype=F32, wdtype=BF16)) == MLP_ERR_INVALID_ARG and "wdtype" in err()
    assert call(desc(dtype=BF16, wdtype=F16)) == MLP_ERR_INVALID_ARG
    assert call(desc(kind=2)) == MLP_ERR_INVALID_ARG and "norm_kind" in err()
    for eps in (-1e-6, math.nan, math.inf):
        assert call(desc(eps=eps)) == MLP_ERR_INVALID_ARG and "eps" in err()
    assert call(desc(M=-1)) == MLP_ERR_INVALID_ARG
    assert call(desc(d=0)) == MLP_ERR_INVALID_ARG
    assert call(desc(d=12)) == MLP_ERR_ALIGNMENT and "multiple of 8" in err()
    assert call(desc(d=10, dtype=F32, wdtype=F32)) == MLP_ERR_ALIGNMENT and "multiple of 4" in err()
    assert call(desc(M=(1 << 30) + 1)) == MLP_ERR_UNSUPPORTED
    assert call(desc(d=1 << 25)) == MLP_ERR_UNSUPPORTED
    assert call(desc(M=1 << 29, d=1 << 20)) == MLP_ERR_UNSUPPORTED


def test_pointer_checks():
    q, rms = desc(), desc(kind=1)
    for n in ("x", "y"):
        assert fwd(q, **{n: None}) == MLP_ERR_INVALID_ARG and n in err()
        assert fwd(q, **{n: FAKE + 8}) == MLP_ERR_ALIGNMENT
    for n in ("res", "w", "b"):
        assert fwd(q, **{n: FAKE + 8}) == MLP_ERR_ALIGNMENT
    for n in ("mean", "rstd"):
        assert fwd(q, **{n: FAKE + 2}) == MLP_ERR_ALIGNMENT
    assert fwd(q, w=None) == MLP_ERR_INVALID_ARG and "weight" in err()
    assert fwd(q, h=FAKE) == MLP_ERR_INVALID_ARG and "residual" in err()
    assert fwd(rms) == MLP_ERR_INVALID_ARG and "mean must be NULL for RMS norm" in err()
    for n in ("dy", "h", "mean", "rstd", "ws"):
        assert bwd(q, **{n: None}) == MLP_ERR_INVALID_ARG, n
    for n in ("dy", "h", "w", "dx", "dw", "db", "dres", "ws"):
        assert bwd(q, **{n: FAKE + 8}) == MLP_ERR_ALIGNMENT, n
    assert bwd(rms) == MLP_ERR_INVALID_ARG and "mean" in err()
    assert bwd(q, dres=FAKE, dx=None) == MLP_ERR_INVALID_ARG and "dx" in err()
    assert bwd(q, acc=2) == MLP_ERR_INVALID_ARG
    assert bwd(q, nws=gm.norm_workspace_bytes(5, 64) - 1) == MLP_ERR_WORKSPACE


def test_nothing_to_do():
    assert fwd(desc(M=0), x=None, y=None) == MLP_OK
    assert bwd(desc(M=0), dy=None, h=None, mean=None, rstd=None, dw=None, db=None) == MLP_OK
    assert bwd(desc(), dx=None, dw=None, db=None, ws=None, nws=0) == MLP_OK


def test_workspaces():
    assert gm.lib().norm_workspace_bytes(-1, 8) == 0 and gm.lib().norm_workspace_bytes(4, 1 << 25) == 0
    with pytest.raises(gm.MlpError, match="2\\^30"):
        gm.norm_workspace_bytes(1 << 31, 8)
    for M in (0, 1, 17, 1024, 1025, 1 << 20):
        for d in (4, 64, 4096, 16384, 16392, 1 << 17):
            assert 256 <= gm.norm_workspace_bytes(M, d) <= max(256, 1024 * 2 * d * 4 + 256)


def test_balance_checks():
    def bal(logits=FAKE, ids=FAKE, mask=None, dtype=BF16, T=5, E=8, k=2, score=0, counts=FAKE, shares=FAKE, loss=FAKE, ws=FAKE,
            nws=1 << 30):
        return gm.lib().moe_balance(logits, ids, mask, dtype, T, E, k, score, counts, shares, loss, ws, nws, None)

    def back(logits=FAKE, ids=FAKE, mask=None, counts=FAKE, dloss=None, dw=FAKE, dtype=BF16, T=5, E=8, k=2, score=0, renorm=1,
             dl=FAKE):
        return gm.lib().moe_balance_bwd(logits, ids, mask, counts, dloss, dw, dtype, T, E, k, score, renorm, dl, None)

    for call in (bal, back):
        assert call(dtype=3) == MLP_ERR_INVALID_ARG
        assert call(T=-1) == MLP_ERR_INVALID_ARG
        assert call(E=1025) == MLP_ERR_UNSUPPORTED
        assert call(k=9) == MLP_ERR_INVALID_ARG
        assert call(score=2) == MLP_ERR_INVALID_ARG
        assert call(T=1 << 30) == MLP_ERR_UNSUPPORTED
        assert call(logits=None) == MLP_ERR_INVALID_ARG and "logits" in err()
        assert call(logits=FAKE + 8) == MLP_ERR_ALIGNMENT
        assert call(ids=FAKE + 2) == MLP_ERR_ALIGNMENT
        assert call(counts=None) == MLP_ERR_INVALID_ARG and "counts" in err()
        assert call(counts=FAKE + 1) == MLP_ERR_ALIGNMENT
    for n in ("shares", "loss", "ws"):
        assert bal(**{n: None}) == MLP_ERR_INVALID_ARG and (n if n != "ws" else "workspace") in err()
    assert bal(nws=gm.moe_balance_workspace_bytes(5, 8) - 1) == MLP_ERR_WORKSPACE
    assert back(renorm=2) == MLP_ERR_INVALID_ARG
    assert back(dl=None) == MLP_ERR_INVALID_ARG
    assert back(dw=FAKE + 2) == MLP_ERR_ALIGNMENT and back(dloss=FAKE + 2) == MLP_ERR_ALIGNMENT
    assert back(T=0, logits=None, ids=None, dl=None) == MLP_OK
    assert gm.lib().moe_balance_workspace_bytes(5, 0) == 0
    for T in (0, 1, 1000, 1 << 20):
        for E in (1, 8, 60, 1024):
            assert 256 <= gm.moe_balance_workspace_bytes(T, E) <= 130 * (2 * E + 1) * 4 + 256


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_tensors_are_checked():
    with pytest.raises(ValueError, match="kind must be one of"):
        gm.norm_fwd(t(3, 16), t(3, 16), kind="batch")
    with pytest.raises(ValueError, match=r"y must be torch.bfloat16 \[3, 16\], not torch.bfloat16 \[3, 8\]"):
        gm.norm_fwd(t(3, 16), t(3, 8))
    with pytest.raises(ValueError, match=r"bias must be torch.float32 \[16\], not torch.bfloat16 \[16\]"):
        gm.norm_fwd(t(3, 16), t(3, 16), weight=t(16, dtype=torch.float32), bias=t(16))
    with pytest.raises(ValueError, match="x must be contiguous"):
        gm.norm_fwd(t(16, 3).t(), t(3, 16))
    with pytest.raises(ValueError, match="x must be a float32, bfloat16 or float16 tensor"):
        gm.norm_fwd(t(3, 16, dtype=torch.float64), t(3, 16, dtype=torch.float64))
    with pytest.raises(ValueError, match="on the GPU"):
        gm.norm_fwd(t(3, 16), t(3, 16))
    s = t(3, dtype=torch.float32)
    with pytest.raises(ValueError, match="dweight must be torch.float32"):
        gm.norm_bwd(t(3, 16), t(3, 16), s, t(3, 16), mean=s, weight=t(16), dweight=t(16), grad_accum=True)
    with pytest.raises(ValueError, match=r"rstd must be torch.float32 \[3\]"):
        gm.norm_bwd(t(3, 16), t(3, 16), t(4, dtype=torch.float32), t(3, 16), mean=s)
    ids, c, f = t(3, 2, dtype=I32), t(9, dtype=I32), t(8, dtype=torch.float32)
    one = t(1, dtype=torch.float32)
    with pytest.raises(ValueError, match=r"counts must be torch.int32 \[9\], not torch.int32 \[8\]"):
        gm.moe_balance(t(3, 8), ids, t(8, dtype=I32), f, one)
    with pytest.raises(ValueError, match=r"mask must be torch.bool \[3\], not torch.uint8 \[3\]"):
        gm.moe_balance(t(3, 8), ids, c, f, one, mask=t(3, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dlogits must be torch.bfloat16"):
        gm.moe_balance_bwd(t(3, 8), ids, c, t(3, 8, dtype=torch.float32))
    with pytest.raises(ValueError, match="score must be one of"):
        gm.moe_balance(t(3, 8), ids, c, f, one, score="tanh")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_reference_gradients_are_differences(kind):
    g = torch.Generator().manual_seed(2)
    h, dy = (torch.randn(5, 24, generator=g, dtype=torch.float64) + 0.3 for _ in range(2))
    w, b = (torch.randn(24, generator=g, dtype=torch.float64) for _ in range(2))
    _, mean, rstd, *_ = N.norm_fwd(h, w, b, kind, 1e-5)
    dx, dw, db, *_ = N.norm_bwd(dy, h, mean, rstd, w, None, kind)
    at = [h, w, b]
    for i, grad in enumerate((dx, dw, db)):
        v = torch.randn(at[i].shape, generator=g, dtype=torch.float64)
        hi, lo = ((N.norm_fwd(*[a + s * 1e-6 * v if j == i else a for j, a in enumerate(at)], kind, 1e-5)[0] * dy).sum() for s in (1, -1))
        assert abs((hi - lo) / 2e-6 - (grad * v).sum()) < 1e-6


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_reference_balance_gradient_is_a_difference(score):
    g = torch.Generator().manual_seed(3)
    x, v = (torch.randn(9, 7, generator=g, dtype=torch.float64) for _ in range(2))
    ids, mask = torch.randint(-1, 8, (9, 3), generator=g), torch.rand(9, generator=g) < 0.7
    counts, _, _ = N.balance(x, ids, mask, score)
    d, _ = N.balance_bwd(x, counts, 3, mask, 1.0, score)
    hi, lo = (N.balance(x + s * 1e-6 * v, ids, mask, score)[2] for s in (1, -1))
    assert abs((hi - lo) / 2e-6 - (d * v).sum()) < 1e-8
