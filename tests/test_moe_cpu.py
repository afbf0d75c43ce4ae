"""CPU tests of the mixture-of-experts entry points: every declared symbol is there, arguments are
refused on the host before any HIP call, workspaces are sized, and the float64 references agree with
differences of themselves. No call below reaches a GPU."""
import ctypes as C
import os
import re

import pytest
import torch

import gated_mlp_gemms_amd as gm
import moe_reference as R
from gated_mlp_gemms_amd import _lib
from gated_mlp_gemms_amd._lib import MLP_ERR_ALIGNMENT, MLP_ERR_INVALID_ARG, MLP_ERR_UNSUPPORTED, MLP_ERR_WORKSPACE, MLP_OK

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000      # 16-byte aligned, never dereferenced: each call fails validation first
BF16 = 1


def err():
    return gm.lib().mlp_last_error().decode()


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b((?:moe|linear)_\w+)\s*\(", text)))
    assert set(names) == set(_lib._MOE_SIGNATURES)
    for n in names:
        assert hasattr(gm.lib(), n), n
    assert gm.lib().moe_abi_version() == 1
    assert (gm.MOE_MAX_EXPERTS, gm.MOE_MAX_CHOICES, gm.LINEAR_ACT_NONE) == (1024, 16, -1)


# ---- C entry points ------------------------------------------------------------------------------

def route(logits=FAKE, dtype=BF16, T=5, E=8, k=2, score=0, renorm=1, ids=FAKE, w=FAKE):
    return gm.lib().moe_route(logits, dtype, T, E, k, score, renorm, ids, w, None)


def route_bwd(logits=FAKE, ids=FAKE, dw=FAKE, dtype=BF16, T=5, E=8, k=2, score=0, renorm=1, dl=FAKE):
    return gm.lib().moe_route_bwd(logits, ids, dw, dtype, T, E, k, score, renorm, dl, None)


@pytest.mark.parametrize("call", [route, route_bwd])
def test_router_checks(call):
    assert call(dtype=3) == MLP_ERR_INVALID_ARG and "dtype" in err()
    assert call(T=-1) == MLP_ERR_INVALID_ARG
    assert call(E=0, k=0) == MLP_ERR_INVALID_ARG
    assert call(E=1025) == MLP_ERR_UNSUPPORTED and "1024" in err()
    assert call(k=0) == MLP_ERR_INVALID_ARG
    assert call(k=9) == MLP_ERR_INVALID_ARG
    assert call(E=64, k=17) == MLP_ERR_UNSUPPORTED and "16" in err()
    assert call(T=(1 << 30) // 2 + 1) == MLP_ERR_UNSUPPORTED
    assert call(T=(1 << 62)) == MLP_ERR_UNSUPPORTED
    assert call(score=2) == MLP_ERR_INVALID_ARG
    assert call(renorm=2) == MLP_ERR_INVALID_ARG
    assert call(logits=None) == MLP_ERR_INVALID_ARG and "logits is NULL" in err()
    assert call(logits=FAKE + 8) == MLP_ERR_ALIGNMENT
    assert call(ids=FAKE + 2) == MLP_ERR_ALIGNMENT
    assert call(T=0, logits=None, ids=None) == MLP_OK


def test_sort_checks():
    def sort(ids=FAKE, n=100, E=8, off=FAKE, row=FAKE, slot=FAKE, ws=FAKE, nws=1 << 20):
        return gm.lib().moe_sort(ids, n, E, off, row, slot, ws, nws, None)

    assert sort(n=-1) == MLP_ERR_INVALID_ARG
    assert sort(n=(1 << 30) + 1) == MLP_ERR_UNSUPPORTED
    assert sort(E=0) == MLP_ERR_INVALID_ARG
    assert sort(E=1025) == MLP_ERR_UNSUPPORTED
    for name in ("ids", "off", "row", "slot"):
        assert sort(**{name: None}) == MLP_ERR_INVALID_ARG
        assert sort(**{name: FAKE + 1}) == MLP_ERR_ALIGNMENT
    assert sort(ws=None) == MLP_ERR_INVALID_ARG
    need = gm.moe_sort_workspace_bytes(100000, 64)
    assert sort(n=100000, E=64, nws=need - 1) == MLP_ERR_WORKSPACE
    assert gm.lib().moe_sort_workspace_bytes(10, 0) == 0
    with pytest.raises(gm.MlpError, match="2\\^30"):
        gm.moe_sort_workspace_bytes(1 << 31, 8)
    for n in (0, 1, 4096, 4097, 1 << 20, 1 << 30):
        assert gm.moe_sort_workspace_bytes(n, 1024) <= 65 * 1025 * 4 + 256




def test_row_checks():
    L = gm.lib()
    dims = dict(dtype=BF16, T=5, E=8, k=2, d=64)

    def gather(x=FAKE, slot=FAKE, off=FAKE, xs=FAKE, **kw):
        v = {**dims, **kw}
        return L.moe_gather(x, slot, off, *v.values(), xs, None)

    def gather_bwd(dxs=FAKE, row=FAKE, off=FAKE, dx=FAKE, **kw):
        v = {**dims, **kw}
        return L.moe_gather_bwd(dxs, row, off, *v.values(), dx, None)

    def combine(ys=FAKE, w=FAKE, row=FAKE, off=FAKE, res=None, out=FAKE, **kw):
        v = {**dims, **kw}
        return L.moe_combine(ys, w, row, off, res, *v.values(), out, None)

    def combine_bwd(dout=FAKE, ys=FAKE, w=FAKE, slot=FAKE, off=FAKE, dys=FAKE, dw=FAKE, **kw):
        v = {**dims, **kw}
        return L.moe_combine_bwd(dout, ys, w, slot, off, *v.values(), dys, dw, None)

    for call, names in ((gather, "x slot off xs"), (gather_bwd, "dxs row off dx"), (combine, "ys w row off out"),
                        (combine_bwd, "dout ys w slot off dys dw")):
        assert call(dtype=9) == MLP_ERR_INVALID_ARG
        assert call(d=0) == MLP_ERR_INVALID_ARG
        assert call(d=68) == MLP_ERR_ALIGNMENT and "multiple of 8" in err()
        assert call(d=66, dtype=0) == MLP_ERR_ALIGNMENT
        assert call(d=1 << 25) == MLP_ERR_UNSUPPORTED
        assert call(T=-3) == MLP_ERR_INVALID_ARG
        assert call(k=9) == MLP_ERR_INVALID_ARG
        assert call(E=2000) == MLP_ERR_UNSUPPORTED
        for n in names.split():
            assert call(**{n: None}) == MLP_ERR_INVALID_ARG, n
            assert call(**{n: FAKE + 2}) == MLP_ERR_ALIGNMENT, n
    assert combine(res=FAKE + 4) == MLP_ERR_ALIGNMENT
    assert gather(T=0, x=None, slot=None, xs=None) == MLP_OK


def desc(M=300, K=264, N=136, act="swiglu", dtype="bf16", experts=0):
    return gm.make_linear_desc(M, K, N, act=act, dtype=dtype, experts=experts)


def fwd(d, x=FAKE, w=FAKE, up=FAKE, b=None, bu=None, res=None, off=None, y=FAKE, pre=None, ws=FAKE, nws=1 << 40):
    return gm.lib().linear_fwd(C.byref(d) if d else None, x, w, up, b, bu, res, off, y, pre, ws, nws, None)


def bwd(d, dy=FAKE, x=FAKE, w=FAKE, up=FAKE, pre=FAKE, off=None, dx=FAKE, dw=FAKE, dwu=FAKE, db=None, dbu=None, acc=0,
        ws=FAKE, nws=1 << 40):
    return gm.lib().linear_bwd(C.byref(d) if d else None, dy, x, w, up, pre, off, dx, dw, dwu, db, dbu, acc, ws, nws, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_linear_descriptor_checks(call):
    assert call(None) == MLP_ERR_INVALID_ARG
    d = desc()
    d.act = 7
    assert call(d) == MLP_ERR_INVALID_ARG
    d.act = -2
    assert call(d) == MLP_ERR_INVALID_ARG
    d = desc()
    d.dtype = 3
    assert call(d) == MLP_ERR_INVALID_ARG
    assert call(desc(M=-1)) == MLP_ERR_INVALID_ARG
    assert call(desc(K=0)) == MLP_ERR_INVALID_ARG
    assert call(desc(N=0)) == MLP_ERR_INVALID_ARG
    assert call(desc(experts=-1)) == MLP_ERR_INVALID_ARG
    assert call(desc(experts=1025)) == MLP_ERR_UNSUPPORTED
    assert call(desc(K=260)) == MLP_ERR_ALIGNMENT and "multiples of 8" in err()
    assert call(desc(N=132)) == MLP_ERR_ALIGNMENT
    assert call(desc(N=130, dtype="f32")) == MLP_ERR_ALIGNMENT
    assert call(desc(M=(1 << 30) + 1)) == MLP_ERR_UNSUPPORTED
    assert call(desc(N=1 << 24)) == MLP_ERR_UNSUPPORTED            # gated: 2N
    assert call(desc(N=1 << 25, act="none"), ) == MLP_ERR_UNSUPPORTED
    assert call(desc(M=1 << 28, K=1 << 20)) == MLP_ERR_UNSUPPORTED
    assert call(desc(M=64, K=1 << 20, N=1 << 20, experts=2)) == MLP_ERR_UNSUPPORTED
    assert call(desc(M=1 << 29, K=8, N=8, experts=1024), off=FAKE) == MLP_ERR_UNSUPPORTED
    assert gm.lib().linear_workspace_bytes(C.byref(desc(K=260)), 0) == 0
    assert gm.lib().linear_workspace_bytes(C.byref(desc()), 2) == 0


def test_linear_pointer_checks():
    d, plain, many = desc(), desc(act="relu"), desc(experts=4)
    for n in ("x", "w", "y", "ws"):
        assert fwd(d, **{n: None}) == MLP_ERR_INVALID_ARG, n
        assert fwd(d, **{n: FAKE + 8}) == MLP_ERR_ALIGNMENT, n
    assert fwd(d, up=None) == MLP_ERR_INVALID_ARG and "w_up" in err()
    assert fwd(plain) == MLP_ERR_INVALID_ARG and "w_up" in err()
    assert fwd(d, b=FAKE) == MLP_ERR_INVALID_ARG and "both" in err()
    assert fwd(plain, up=None, b=FAKE, bu=FAKE) == MLP_ERR_INVALID_ARG and "bias_up" in err()
    assert fwd(d, off=FAKE) == MLP_ERR_INVALID_ARG and "offsets" in err()
    assert fwd(many) == MLP_ERR_INVALID_ARG and "offsets" in err()
    for n in ("res", "pre"):
        assert fwd(d, **{n: FAKE + 2}) == MLP_ERR_ALIGNMENT
    assert fwd(d, nws=255) == MLP_ERR_WORKSPACE

    for n in ("dy", "x", "w", "pre", "ws"):
        assert bwd(d, **{n: None}) == MLP_ERR_INVALID_ARG, n
        assert bwd(d, **{n: FAKE + 8}) == MLP_ERR_ALIGNMENT, n
    assert bwd(d, dwu=None) == MLP_ERR_INVALID_ARG and "both" in err()
    assert bwd(d, db=FAKE) == MLP_ERR_INVALID_ARG and "both" in err()
    assert bwd(plain, up=None) == MLP_ERR_INVALID_ARG and "dw_up" in err()
    assert bwd(plain, up=None, dwu=None, db=FAKE, dbu=FAKE) == MLP_ERR_INVALID_ARG and "dbias_up" in err()
    assert bwd(desc(act="none"), up=None, dwu=None) == MLP_ERR_INVALID_ARG and "preact" in err()
    assert bwd(d, acc=2) == MLP_ERR_INVALID_ARG
    assert bwd(many) == MLP_ERR_INVALID_ARG and "offsets" in err()
    need = gm.linear_workspace_bytes(d, "bwd")
    assert need >= 300 * 2 * 136 * 2 and bwd(d, nws=need - 1) == MLP_ERR_WORKSPACE


def test_linear_of_nothing_and_nothing_asked_for():
    assert fwd(desc(M=0), x=None, y=None) == MLP_OK
    assert bwd(desc(M=0), dy=None, x=None, pre=None, dx=None, dw=None, dwu=None) == MLP_OK


def test_workspaces_over_a_grid():
    """Every size the descriptor allows plans without trouble (a few rows to the limits)."""
    for act in ("none", "gelu_tanh", "swiglu"):
        for dt in ("bf16", "f32"):
            for M in (0, 1, 16, 17, 300, 5000, 1 << 20):
                for K, N in ((8, 8), (264, 136), (4096, 11008), (8192, 64)):
                    for E in (0, 1, 7, 1024):
                        d = desc(M=M, K=K, N=N, act=act, dtype=dt, experts=E)
                        assert gm.linear_workspace_bytes(d, "fwd") >= 256
                        assert gm.linear_workspace_bytes(d, "bwd") >= 256


# ---- Python side: tensors ------------------------------------------------------------------------

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


I32, F32 = torch.int32, torch.float32


def test_tensors_are_checked():
    ids, w = t(5, 2, dtype=I32), t(5, 2, dtype=F32)
    bad = [
        (lambda: gm.moe_route(t(5, 8), ids, w), "GPU"),
        (lambda: gm.moe_route(t(5, 8), ids.long(), w), "ids must be torch.int32"),
        (lambda: gm.moe_route(t(5, 8), ids, w.bfloat16()), "weights must be"),
        (lambda: gm.moe_route(t(5, 8), ids, t(4, 2, dtype=F32)), "weights must be"),
        (lambda: gm.moe_route(t(8, 5).t(), ids, w), "contiguous"),
        (lambda: gm.moe_route(t(5, 8, dtype=torch.float64), ids, w), "logits must be"),
        (lambda: gm.moe_route(t(40), ids, w), "2 dimensions"),
        (lambda: gm.moe_route(None, ids, w), "logits"),
        (lambda: gm.moe_route(t(5, 8), ids, w, score="max"), "score"),
        (lambda: gm.moe_route_bwd(t(5, 8), ids, w, t(5, 8, dtype=F32)), "dlogits"),
        (lambda: gm.moe_sort(ids, 8, t(8, dtype=I32), t(10, dtype=I32), t(10, dtype=I32)), "offsets"),
        (lambda: gm.moe_sort(ids, 8, t(9, dtype=I32), t(10, dtype=I32), t(10, dtype=I32)), "GPU"),
        (lambda: gm.moe_gather(t(5, 64), t(10, dtype=I32), t(9, dtype=I32), t(11, 64)), "not a multiple"),
        (lambda: gm.moe_gather(t(5, 64), t(10, dtype=I32), t(9, dtype=I32), t(10, 32)), "xs"),
        (lambda: gm.moe_combine(t(10, 64), w, t(10, dtype=I32), t(9, dtype=I32), t(5, 64), residual=t(5, 32)), "residual"),
        (lambda: gm.moe_combine_bwd(t(5, 64), t(10, 64), w, t(9, dtype=I32), t(10, dtype=I32), t(9, dtype=I32), t(10, 64),
                                    w), "row_of"),
        (lambda: gm.moe_gather_bwd(t(10, 64), t(10, dtype=I32), t(9, dtype=I32), t(5, 64, dtype=F32)), "dxs"),
    ]
    d = desc(M=6, K=16, N=24, experts=3)
    good = dict(w_up=t(3, 24, 16), offsets=t(4, dtype=I32))
    bad += [
        (lambda: gm.linear_fwd(d, t(6, 16), t(3, 24, 16), t(6, 24), **good), "GPU"),
        (lambda: gm.linear_fwd(d, t(6, 16), t(24, 16), t(6, 24), **good), "w must be"),
        (lambda: gm.linear_fwd(d, t(6, 16), t(3, 24, 16), t(6, 24), **{**good, "offsets": t(3, dtype=I32)}), "offsets"),
        (lambda: gm.linear_fwd(d, t(6, 16), t(3, 24, 16), t(6, 24), preact=t(6, 24), **good), "preact"),
        (lambda: gm.linear_fwd(d, t(6, 32)[:, ::2], t(3, 24, 16), t(6, 24), **good), "contiguous"),
        (lambda: gm.linear_bwd(d, t(6, 24), t(6, 16), t(3, 24, 16), preact=t(6, 48), dw=t(3, 24, 16), dw_up=t(3, 24, 16),
                               grad_accum=True, **good), "dw must be torch.float32"),
        (lambda: gm.linear_bwd(d, t(6, 24), t(6, 16), t(3, 24, 16), preact=t(6, 48), dbias=t(24), **good), "dbias"),
    ]
    for call, text in bad:
        with pytest.raises(ValueError, match=text):
            call()


# ---- the references themselves --------------------------------------------------------------------

@pytest.mark.parametrize("act", R.ACTS)
def test_reference_gradients_are_differences(act):
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)   # noqa: E731
    M, K, N, E = 7, 5, 4, 3
    off = torch.tensor([0, 3, 3, 6])
    x, w, wu, b, bu, dy = rnd(M, K), rnd(E, N, K), rnd(E, N, K), rnd(E, N), rnd(E, N), rnd(M, N)
    dy[6:] = 0
    loss = lambda: (R.linear(act, x, w, wu, b, bu, None, off)[0] * dy).sum()   # noqa: E731
    _, pre, _ = R.linear(act, x, w, wu, b, bu, None, off)
    r = R.linear_bwd(act, dy, x, w, wu, pre, off)
    pairs = [(x, r["dx"][0]), (w, r["dw"][0][0]), (b, r["db"][0][0])]
    if act in R.GATED:
        pairs += [(wu, r["dw"][1][0]), (bu, r["db"][1][0])]
    h = 1e-6
    for leaf, grad in pairs:
        v = rnd(*leaf.shape)
        leaf += h * v
        hi = loss()
        leaf -= 2 * h * v
        lo = loss()
        leaf += h * v
        assert abs((hi - lo) / (2 * h) - (grad * v).sum()) < 1e-6


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_router_gradient_is_a_difference(score, renorm):
    g = torch.Generator().manual_seed(4)
    x, dw, v = (torch.randn(6, n, generator=g, dtype=torch.float64) for n in (9, 3, 9))
    ids = R.route(x, 3, score, renorm)[0]

    def loss(z):
        _, _, p = R.route(z, 3, score, renorm)
        w = p.gather(1, ids)
        w = w / w.sum(dim=1, keepdim=True) if renorm else w
        return (w * dw).sum()

    h = 1e-6
    assert abs((loss(x + h * v) - loss(x - h * v)) / (2 * h) - (R.route_bwd(x, ids, dw, score, renorm) * v).sum()) < 1e-8


# ---- the binding ----------------------------------------------------------------------------------

def test_binding_refuses_what_is_not_a_tensor_or_descriptor():
    b = _lib.bind()
    with pytest.raises(TypeError, match="6 arguments expected, not 2"):
        b.moe_route(t(5, 8), t(5, 2, dtype=I32))
    with pytest.raises(ValueError, match="weights must be a tensor, not list"):
        gm.moe_route(t(5, 8), t(5, 2, dtype=I32), [1.0])
    with pytest.raises(ValueError, match=r"weights must be torch.float32 \[5, 2\], not torch.bfloat16 \[5, 3\]"):
        gm.moe_route(t(5, 8), t(5, 2, dtype=I32), t(5, 3))
    with pytest.raises(ValueError, match=r"logits must be contiguous, not of strides \[1, 5\]"):
        gm.moe_route(t(8, 5).t(), t(5, 2, dtype=I32), t(5, 2, dtype=F32))
    with pytest.raises(ValueError, match="logits must be on the GPU of the other tensors, not on cpu"):
        gm.moe_route(t(5, 8), t(5, 2, dtype=I32), t(5, 2, dtype=F32))
    with pytest.raises(ValueError, match="contiguous"):
        gm.moe_sort(t(4, 2, dtype=I32).t(), 3, t(4, dtype=I32), t(8, dtype=I32), t(8, dtype=I32))
    with pytest.raises(ValueError, match="ids must be a tensor"):
        gm.moe_sort(None, 3, t(4, dtype=I32), t(8, dtype=I32), t(8, dtype=I32))
    with pytest.raises(TypeError):
        gm.moe_sort(t(8, dtype=I32), "3", t(4, dtype=I32), t(8, dtype=I32), t(8, dtype=I32))
    with pytest.raises(ValueError, match="LinearDesc"):
        gm.linear_fwd(b"x", t(6, 16), t(24, 16), t(6, 24))
    with pytest.raises(TypeError):
        gm.linear_fwd(None, t(6, 16), t(24, 16), t(6, 24))
    with pytest.raises(ValueError, match="x must be contiguous"):
        gm.linear_fwd(desc(M=6, K=16, N=24, act="none"), t(6, 16).to_sparse(), t(24, 16), t(6, 24))


def test_binding_is_required(monkeypatch):
    monkeypatch.setattr(_lib, "_bind", None)
    monkeypatch.setitem(__import__("sys").modules, "gated_mlp_gemms_amd._bind", None)
    monkeypatch.delattr(gm, "_bind", raising=False)
    with pytest.raises(RuntimeError, match="_bind extension"):
        gm.moe_route(t(5, 8), t(5, 2, dtype=I32), t(5, 2, dtype=F32))


def test_rows_beyond_a_launch_are_refused():
    assert fwd(desc(M=(1 << 29) + 8, K=8, N=8)) == MLP_ERR_UNSUPPORTED and "2^29" in err()
    assert gm.linear_workspace_bytes(desc(M=1 << 29, K=8, N=8, act="none"), "bwd") >= 256
