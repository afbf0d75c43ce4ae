"""CPU tests of the 4-bit entry points: every declared symbol is there, arguments are refused on the host before any
HIP call, workspaces are sized, and the references agree with the format's definition. No call below reaches a GPU."""
import ctypes as C
import math
import os
import re

import pytest
import torch

import gated_mlp_gemms_amd as gm
import mx4_reference as X
from gated_mlp_gemms_amd import _lib
from gated_mlp_gemms_amd._lib import MLP_ERR_ALIGNMENT, MLP_ERR_INVALID_ARG, MLP_ERR_UNSUPPORTED, MLP_ERR_WORKSPACE, MLP_OK

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000      # 16-byte aligned, never dereferenced: each call fails validation first
F32, BF16 = 0, 1
U8 = torch.uint8


def err():
    return gm.lib().mlp_last_error().decode()


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mx4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(mx4_\w+)\s*\(", text))
    assert names == set(_lib._MX4_SIGNATURES)
    for n in names:
        assert hasattr(gm.lib(), n), n


def test_shapes():
    assert gm.mx4_shapes(5, 64) == ((5, 32), (1, 8, 8))
    assert gm.mx4_shapes(8, 544, batch=3) == ((3, 8, 272), (3, 3, 12, 8))
    assert gm.mx4_shapes(0, 32) == ((0, 16), (1, 4, 8))
    assert gm.lib().mx4_planes(-1) == 0 and gm.lib().mx4_scale_rows(-1) == 0


def quantize(x=FAKE, dtype=BF16, batch=1, rows=5, cols=64, c=FAKE, s=FAKE, ct=FAKE, st=FAKE):
    return gm.lib().mx4_quantize(x, dtype, batch, rows, cols, c, s, ct, st, None)


def dequantize(c=FAKE, s=FAKE, dtype=BF16, batch=1, rows=5, cols=64, out=FAKE):
    return gm.lib().mx4_dequantize(c, s, dtype, batch, rows, cols, out, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_matrix_checks(call):
    assert call(dtype=3) == MLP_ERR_INVALID_ARG and "dtype" in err()
    assert call(rows=-1) == MLP_ERR_INVALID_ARG
    assert call(cols=0) == MLP_ERR_INVALID_ARG
    assert call(batch=-1) == MLP_ERR_INVALID_ARG
    assert call(batch=65536) == MLP_ERR_UNSUPPORTED
    assert call(rows=(1 << 29) + 1) == MLP_ERR_UNSUPPORTED
    assert call(cols=1 << 25) == MLP_ERR_UNSUPPORTED
    assert call(rows=1 << 28, cols=1 << 20) == MLP_ERR_UNSUPPORTED
    assert call(cols=48) == MLP_ERR_ALIGNMENT and "32" in err()
    for n in ("c", "s"):
        assert call(**{n: None}) == MLP_ERR_INVALID_ARG, n
        assert call(**{n: FAKE + 8}) == MLP_ERR_ALIGNMENT, n


def test_quantize_checks():
    assert quantize(x=None) == MLP_ERR_INVALID_ARG and quantize(x=FAKE + 8) == MLP_ERR_ALIGNMENT
    assert quantize(ct=None) == MLP_ERR_INVALID_ARG and "codes_t" in err()
    assert quantize(st=FAKE + 4) == MLP_ERR_ALIGNMENT
    assert quantize(cols=36, c=None, s=None) == MLP_ERR_ALIGNMENT and "multiple of 8" in err()
    assert quantize(cols=34, c=None, s=None, dtype=F32) == MLP_ERR_ALIGNMENT and "multiple of 4" in err()
    assert quantize(c=None, s=None, ct=None, st=None) == MLP_OK
    assert quantize(rows=0, x=None, c=None, s=None, ct=None, st=None) == MLP_OK
    assert dequantize(rows=0, c=None, s=None, out=None) == MLP_OK
    assert dequantize(out=None) == MLP_ERR_INVALID_ARG


def desc(M=300, K=256, N=136, act="swiglu", dtype="bf16", experts=0):
    return gm.make_linear_desc(M, K, N, act=act, dtype=dtype, experts=experts)


def fwd(d, x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, up=FAKE, ups=FAKE, b=None, bu=None, res=None, off=None, y=FAKE, pre=None, wk=FAKE, nwk=1 << 40):
    return gm.lib().mx4_linear_fwd(C.byref(d) if d else None, x, xs, w, ws, up, ups, b, bu, res, off, y, pre, wk, nwk, None)


def test_product_descriptor_checks():
    assert fwd(None) == MLP_ERR_INVALID_ARG and "desc is NULL" in err()
    d = desc()
    d.dtype = 3
    assert fwd(d) == MLP_ERR_INVALID_ARG
    d = desc()
    d.act = 9
    assert fwd(d) == MLP_ERR_INVALID_ARG
    assert fwd(desc(M=-1)) == MLP_ERR_INVALID_ARG
    assert fwd(desc(K=0)) == MLP_ERR_INVALID_ARG
    assert fwd(desc(experts=-1)) == MLP_ERR_INVALID_ARG
    assert fwd(desc(experts=1025)) == MLP_ERR_UNSUPPORTED
    assert fwd(desc(K=48)) == MLP_ERR_ALIGNMENT and "32" in err()
    assert fwd(desc(N=132)) == MLP_ERR_ALIGNMENT
    assert fwd(desc(N=132, dtype="f32")) == MLP_ERR_ALIGNMENT and "multiple of 8" in err()
    assert fwd(desc(M=(1 << 29) + 1)) == MLP_ERR_UNSUPPORTED
    assert fwd(desc(N=1 << 24)) == MLP_ERR_UNSUPPORTED
    assert fwd(desc(M=1 << 28, K=1 << 20)) == MLP_ERR_UNSUPPORTED
    assert fwd(desc(M=64, K=1 << 20, N=1 << 20, experts=2)) == MLP_ERR_UNSUPPORTED
    assert gm.lib().mx4_linear_workspace_bytes(C.byref(desc(K=40))) == 0
    with pytest.raises(gm.MlpError, match="multiple of 32"):
        gm.mx4_linear_workspace_bytes(desc(K=40))


def test_product_pointer_checks():
    d, plain, many = desc(), desc(act="relu"), desc(experts=4)
    for n in ("x", "xs", "w", "ws", "up", "ups", "y", "wk"):
        assert fwd(d, **{n: None}) == MLP_ERR_INVALID_ARG, n
        assert fwd(d, **{n: FAKE + 8}) == MLP_ERR_ALIGNMENT, n
    assert fwd(plain) == MLP_ERR_INVALID_ARG and "w_up" in err()
    assert fwd(plain, up=None) == MLP_ERR_INVALID_ARG and "w_up_scales" in err()
    assert fwd(plain, up=None, ups=None, bu=FAKE) == MLP_ERR_INVALID_ARG and "bias_up" in err()
    assert fwd(d, b=FAKE) == MLP_ERR_INVALID_ARG and "both" in err()
    assert fwd(d, off=FAKE) == MLP_ERR_INVALID_ARG and "offsets" in err()
    assert fwd(many) == MLP_ERR_INVALID_ARG and "offsets" in err()
    assert fwd(many, off=FAKE + 2) == MLP_ERR_ALIGNMENT
    for n in ("res", "pre"):
        assert fwd(d, **{n: FAKE + 2}) == MLP_ERR_ALIGNMENT
    assert fwd(d, nwk=255) == MLP_ERR_WORKSPACE
    split = desc(M=17, K=1 << 16, N=64, act="none")
    assert fwd(split, up=None, ups=None, nwk=gm.mx4_linear_workspace_bytes(split) - 1) == MLP_ERR_WORKSPACE
    assert fwd(desc(M=0), x=None, xs=None, y=None) == MLP_OK


def test_workspaces_over_a_grid():
    for act in ("none", "swiglu"):
        for dt in ("bf16", "f32"):
            for M in (0, 1, 16, 17, 300, 5000, 1 << 20):
                for K, N in ((32, 8), (288, 136), (4096, 11008), (8192, 64)):
                    for E in (0, 1, 7, 1024):
                        assert gm.mx4_linear_workspace_bytes(desc(M=M, K=K, N=N, act=act, dtype=dt, experts=E)) >= 256


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def u(shape):
    return torch.zeros(*shape, dtype=U8)


def test_tensors_are_checked():
    c, s = (u(v) for v in gm.mx4_shapes(6, 64))
    with pytest.raises(ValueError, match=r"codes must be torch.uint8 \[6, 32\]"):
        gm.mx4_quantize(t(6, 64), u((6, 64)), s)
    with pytest.raises(ValueError, match=r"scales must be torch.uint8 \[1, 8, 8\], not torch.uint8 \[8, 8\]"):
        gm.mx4_quantize(t(6, 64), c, u((8, 8)))
    with pytest.raises(ValueError, match=r"codes_t must be torch.uint8 \[64, 16\]"):
        gm.mx4_quantize(t(6, 64), codes_t=c, scales_t=s)
    with pytest.raises(ValueError, match="x must be a tensor of 2 dimensions"):
        gm.mx4_quantize(t(64), c, s)
    with pytest.raises(ValueError, match="on the GPU"):
        gm.mx4_quantize(t(6, 64), c, s)
    with pytest.raises(ValueError, match="x must be contiguous"):
        gm.mx4_quantize(t(64, 6).t(), c, s)
    with pytest.raises(ValueError, match="out must be a float32, bfloat16 or float16 tensor"):
        gm.mx4_dequantize(c, s, t(6, 64, dtype=torch.int32))
    wc, ws = (u(v) for v in gm.mx4_shapes(24, 64))
    d = desc(M=6, K=64, N=24, act="none")
    with pytest.raises(ValueError, match=r"w_scales must be torch.uint8 \[1, 28, 8\]"):
        gm.mx4_linear_fwd(d, c, s, wc, s, t(6, 24))
    with pytest.raises(ValueError, match=r"y must be torch.bfloat16 \[6, 24\]"):
        gm.mx4_linear_fwd(d, c, s, wc, ws, t(6, 24, dtype=torch.float32))
    with pytest.raises(ValueError, match="LinearDesc"):
        gm.mx4_linear_fwd(b"x", c, s, wc, ws, t(6, 24))
    many = desc(M=6, K=64, N=24, act="none", experts=3)
    with pytest.raises(ValueError, match=r"w must be torch.uint8 \[3, 24, 32\]"):
        gm.mx4_linear_fwd(many, c, s, wc, ws, t(6, 24))


def test_reference_codes():
    """The reference against the format's own words: a code is the nearest of the grid, ties to the even one."""
    v = torch.tensor([0.0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 1.74, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 7.9, -0.25, -0.75,
                      -0.0, -5.0, -7.0] + [0.0] * 10 + [4.0])
    code, scale = X.encode(v)
    assert scale.tolist() == [127]
    want = [0, 0, 1, 2, 1, 2, 3, 4, 3, 4, 5, 6, 5, 6, 7, 7, 8, 10, 8, 14, 15] + [0] * 10 + [6]
    assert code.tolist() == want
    for top, s in ((1.0, 125), (7.99, 127), (8.0, 128), (0.0, 0), (2.0 ** -126, 0), (2.0 ** -124, 1), (3e38, 252), (math.inf, 255), (math.nan, 255)):
        b = torch.zeros(32)
        b[3] = top
        assert X.encode(b)[1].tolist() == [s], top
    x = torch.randn(6, 96)
    code, scale = X.encode(x)
    back, s = X.unpack(*X.pack(code, scale))
    assert torch.equal(back, code) and torch.equal(s[:, :3], scale)
    # each value within half a step of itself: 1/4 of its power of two, or of the block's smallest step
    big = x.double().reshape(6, 3, 32).abs().amax(-1, keepdim=True).expand(6, 3, 32).reshape(6, 96)
    assert ((X.rounded(x) - x.double()).abs() <= torch.maximum(x.double().abs() / 4, big / 16)).all()


def test_more_threads_than_a_launch_has():
    """Few rows of many experts by a very wide weight: refused, not left to the launch."""
    d = desc(M=8192, K=32, N=1 << 22, act="none", experts=1024)
    assert fwd(d, up=None, ups=None, off=FAKE) == MLP_ERR_UNSUPPORTED and "threads" in err()
