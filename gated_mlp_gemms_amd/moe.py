"""The mixture-of-experts operators of ``include/moe.h``: router, tokens sorted by expert and back,
linear layer with its epilogue, experts' products, and their gradients.

As in the rest of the package the functions carry the C entry points' names, write into buffers the
caller passes, take a workspace (or allocate one with torch) and run on the current stream of their
tensors' device unless ``stream`` is given. Sizes come from the tensors, so every tensor's dtype, shape
and layout (contiguous, on one GPU) is checked first (``ValueError``); what the library refuses raises
``MlpError``. One training step of a layer of E experts, k a token::

    moe_route(logits, ids, weights)                                    # [T, E] -> [T, k]
    moe_sort(ids, E, offsets, row_of, slot_of)
    moe_gather(x, slot_of, offsets, xs)                                # [T, d] -> [T k, d]
    linear_fwd(up, xs, w_gate, a, w_up=w_up, offsets=offsets, preact=pre)
    linear_fwd(down, a, w_down, ys, offsets=offsets)
    moe_combine(ys, weights, row_of, offsets, out, residual=x)

and back: ``moe_combine_bwd``, ``linear_bwd`` twice, ``moe_gather_bwd``, ``moe_route_bwd``.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _ACTS, _DTYPES, GATED_ACTS
from ._lib import (LINEAR_ACT_NONE, LINEAR_BWD, LINEAR_FWD, MOE_SIGMOID, MOE_SOFTMAX, LinearDesc, MlpError, check, lib)

_SCORES = {"softmax": MOE_SOFTMAX, "sigmoid": MOE_SIGMOID}
_PHASES = {"fwd": LINEAR_FWD, "bwd": LINEAR_BWD}
_LINEAR_ACTS = {"none": LINEAR_ACT_NONE, **_ACTS}
_ACT_NAMES = {v: k for k, v in _LINEAR_ACTS.items()}
_TORCH = {v: k for k, v in _DTYPES.items() if isinstance(k, torch.dtype)}
_I32, _F32 = torch.int32, torch.float32


def _bad(t, name, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, not {type(t).__name__}")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, not of strides {t.stride()}")
    raise ValueError(f"{name} must be on the GPU of the other tensors, not on {t.device}")


def _stream(dev, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)   # current_stream(dev) without making a Stream: 1 us less
    return stream if isinstance(stream, int) else stream.cuda_stream


class _Args:
    """Checks a call's tensors and turns them into device pointers. The first one sets the device; a
    call's tensors are looked at completely before its GPU is required."""
    __slots__ = ("dev", "far")

    def __init__(self):
        self.dev, self.far = None, None

    def __call__(self, t, name, dtype, shape):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
            _bad(t, name, dtype, shape)
        dev = t.get_device()
        if self.dev is None:
            self.dev = dev
        if dev < 0 or dev != self.dev:
            self.far = self.far or (t, name, dtype, shape)
        return t.data_ptr()

    def opt(self, t, name, dtype, shape):
        return None if t is None else self(t, name, dtype, shape)

    def stream(self, stream):
        if self.far is not None:
            _bad(*self.far)
        return _stream(self.dev, stream)

    def workspace(self, ws, need):
        """(tensor that keeps it alive, address, bytes) of the caller's workspace, or of a new one."""
        if self.far is not None:
            _bad(*self.far)
        if ws is None:
            ws = torch.empty(need(), dtype=torch.uint8, device=torch.device("cuda", self.dev))
        elif not ws.is_contiguous() or ws.get_device() != self.dev:
            raise ValueError("workspace must be contiguous and on the GPU of the other tensors")
        return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _dtype(t, name):
    code = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise ValueError(f"{name} must be a float32, bfloat16 or float16 tensor")
    return t.dtype, code


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a tensor of {n} dimensions")
    return t.shape


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    return _SCORES[score]


# ---- router --------------------------------------------------------------------------------------

def moe_route(logits, ids, weights, score="softmax", renorm=True, stream=None):
    """The k largest of each token's E scores (``logits`` [T, E], f32 / bf16 / f16), largest first and
    ties to the lowest expert, into ``ids`` [T, k] (int32), and their probabilities into ``weights``
    [T, k] (fp32): ``score`` "softmax" over all experts or each one's "sigmoid", divided by the chosen
    ones' sum with ``renorm``. Scores of -inf are chosen last, with weight 0."""
    a = _Args()
    dt, code = _dtype(logits, "logits")
    T, E = _dims(logits, "logits", 2)
    k = _dims(ids, "ids", 2)[1]
    p = (a(logits, "logits", dt, (T, E)), code, T, E, k, _score(score), int(bool(renorm)), a(ids, "ids", _I32, (T, k)),
         a(weights, "weights", _F32, (T, k)))
    check(lib().moe_route(*p, a.stream(stream)), "moe_route")
    return ids, weights


def moe_route_bwd(logits, ids, dweights, dlogits, score="softmax", renorm=True, stream=None):
    """``dlogits`` [T, E] (logits' dtype): the gradient of :func:`moe_route`'s weights against
    ``dweights`` [T, k] (fp32), ``ids`` being what it chose."""
    a = _Args()
    dt, code = _dtype(logits, "logits")
    T, E = _dims(logits, "logits", 2)
    k = _dims(ids, "ids", 2)[1]
    p = (a(logits, "logits", dt, (T, E)), a(ids, "ids", _I32, (T, k)), a(dweights, "dweights", _F32, (T, k)), code, T,
         E, k, _score(score), int(bool(renorm)), a(dlogits, "dlogits", dt, (T, E)))
    check(lib().moe_route_bwd(*p, a.stream(stream)), "moe_route_bwd")
    return dlogits


# ---- tokens by expert and back -------------------------------------------------------------------

def moe_sort_workspace_bytes(n, experts) -> int:
    b = lib().moe_sort_workspace_bytes(int(n), int(experts))
    if b == 0:
        raise MlpError(1, "moe_sort_workspace_bytes")
    return int(b)


def moe_sort(ids, experts, offsets, row_of, slot_of, workspace=None, stream=None):
    """Slots (the n entries of ``ids``, int32 of any shape) in expert order, stably: ``offsets``
    [experts + 1], ``slot_of`` [n] = the slot in each row, ``row_of`` [n] its inverse, all int32. An id
    outside [0, experts) is dropped: its slot goes behind ``offsets[experts]``."""
    a = _Args()
    n, E = ids.numel() if isinstance(ids, torch.Tensor) else 0, int(experts)
    pi = a(ids, "ids", _I32, ids.shape if isinstance(ids, torch.Tensor) else (n,))
    p = (pi, n, E, a(offsets, "offsets", _I32, (E + 1,)), a(row_of, "row_of", _I32, (n,)),
         a(slot_of, "slot_of", _I32, (n,)))
    keep, ws, nws = a.workspace(workspace, lambda: moe_sort_workspace_bytes(n, E))
    check(lib().moe_sort(*p, ws, nws, a.stream(stream)), "moe_sort")
    return offsets, row_of, slot_of


def _rows(tokens, name, sorted_, sorted_name, offsets, a):
    """(dtype, code, T, E, k, d) of a [T, d] and a [T k, d] tensor, with both checked."""
    dt, code = _dtype(tokens, name)
    T, d = _dims(tokens, name, 2)
    n = _dims(sorted_, sorted_name, 2)[0]
    E = _dims(offsets, "offsets", 1)[0] - 1
    if (n % T if T else n) != 0:
        raise ValueError(f"{sorted_name} has {n} rows, not a multiple of the {T} tokens")
    return dt, code, T, E, n // T if T else 1, d


def moe_gather(x, slot_of, offsets, xs, stream=None):
    """``xs`` [T k, d]: row r is the row of ``x`` [T, d] that slot ``slot_of[r]`` belongs to; zeros
    behind ``offsets[E]``."""
    a = _Args()
    dt, code, T, E, k, d = _rows(x, "x", xs, "xs", offsets, a)
    p = (a(x, "x", dt, (T, d)), a(slot_of, "slot_of", _I32, (T * k,)), a(offsets, "offsets", _I32, (E + 1,)), code, T,
         E, k, d, a(xs, "xs", dt, (T * k, d)))
    check(lib().moe_gather(*p, a.stream(stream)), "moe_gather")
    return xs


def moe_gather_bwd(dxs, row_of, offsets, dx, stream=None):
    """``dx`` [T, d]: each token's sum of its kept rows of ``dxs`` [T k, d], in fp32."""
    a = _Args()
    dt, code, T, E, k, d = _rows(dx, "dx", dxs, "dxs", offsets, a)
    p = (a(dxs, "dxs", dt, (T * k, d)), a(row_of, "row_of", _I32, (T * k,)), a(offsets, "offsets", _I32, (E + 1,)),
         code, T, E, k, d, a(dx, "dx", dt, (T, d)))
    check(lib().moe_gather_bwd(*p, a.stream(stream)), "moe_gather_bwd")
    return dx


def moe_combine(ys, weights, row_of, offsets, out, residual=None, stream=None):
    """``out`` [T, d] = ``residual`` + each token's kept rows of ``ys`` [T k, d] by ``weights`` [T, k]
    (fp32), summed in fp32 and rounded once. ``out`` may be ``residual``."""
    a = _Args()
    dt, code, T, E, k, d = _rows(out, "out", ys, "ys", offsets, a)
    p = (a(ys, "ys", dt, (T * k, d)), a(weights, "weights", _F32, (T, k)), a(row_of, "row_of", _I32, (T * k,)),
         a(offsets, "offsets", _I32, (E + 1,)), a.opt(residual, "residual", dt, (T, d)), code, T, E, k, d,
         a(out, "out", dt, (T, d)))
    check(lib().moe_combine(*p, a.stream(stream)), "moe_combine")
    return out


def moe_combine_bwd(dout, ys, weights, row_of, slot_of, offsets, dys, dweights, stream=None):
    """Both gradients of :func:`moe_combine` against ``dout`` [T, d]: ``dys`` [T k, d] (zeros in the
    dropped rows) and ``dweights`` [T, k] (fp32, 0 for a dropped slot). The residual's is ``dout``.
    It goes by rows and reads ``slot_of``; ``row_of``, its inverse, is only checked."""
    a = _Args()
    dt, code, T, E, k, d = _rows(dout, "dout", ys, "ys", offsets, a)
    n = T * k
    a(row_of, "row_of", _I32, (n,))
    p = (a(dout, "dout", dt, (T, d)), a(ys, "ys", dt, (n, d)), a(weights, "weights", _F32, (T, k)),
         a(slot_of, "slot_of", _I32, (n,)), a(offsets, "offsets", _I32, (E + 1,)), code, T, E, k, d,
         a(dys, "dys", dt, (n, d)), a(dweights, "dweights", _F32, (T, k)))
    check(lib().moe_combine_bwd(*p, a.stream(stream)), "moe_combine_bwd")
    return dys, dweights


# ---- linear layer and the experts' products ------------------------------------------------------

def make_linear_desc(M, K, N, act="none", dtype=torch.bfloat16, experts=0) -> LinearDesc:
    """x [M, K] -> y [M, N]; ``act`` "none" or one of the MLP's activations (a gated one takes a second
    weight); ``experts`` 0: one weight [N, K], else [experts, N, K] and rows grouped by offsets."""
    return LinearDesc(int(M), int(K), int(N), _LINEAR_ACTS[act], _DTYPES[dtype], int(experts))


def linear_workspace_bytes(desc: LinearDesc, phase: str) -> int:
    n = lib().linear_workspace_bytes(C.byref(desc), _PHASES[phase])
    if n == 0:
        raise MlpError(1, "linear_workspace_bytes")
    return int(n)


def _linear_shapes(desc):
    """(dtype, gated, shape of a weight, shape of a bias, columns of preact)"""
    gated = _ACT_NAMES.get(desc.act) in GATED_ACTS
    lead = (desc.experts,) if desc.experts else ()
    dt = _TORCH.get(desc.dtype, _F32)   # (the library refuses another)
    return dt, gated, lead + (desc.N, desc.K), lead + (desc.N,), 2 * desc.N if gated else desc.N


def linear_fwd(desc, x, w, y, w_up=None, bias=None, bias_up=None, residual=None, offsets=None, preact=None,
               workspace=None, stream=None):
    """``y`` [M, N] = residual + act(x w^T + bias), gated: act(x w^T + bias) (x w_up^T + bias_up).
    With experts, row r of ``x`` is of the expert e with offsets[e] <= r < offsets[e + 1]. ``preact``
    receives what the activation was taken of ([M, N], gated [M, 2N] = [g | u]), for linear_bwd."""
    a = _Args()
    dt, _, ws_, bs, P = _linear_shapes(desc)
    M, K, N = desc.M, desc.K, desc.N
    p = (a(x, "x", dt, (M, K)), a(w, "w", dt, ws_), a.opt(w_up, "w_up", dt, ws_), a.opt(bias, "bias", dt, bs),
         a.opt(bias_up, "bias_up", dt, bs), a.opt(residual, "residual", dt, (M, N)),
         a.opt(offsets, "offsets", _I32, (desc.experts + 1,)), a(y, "y", dt, (M, N)),
         a.opt(preact, "preact", dt, (M, P)))
    keep, ws, nws = a.workspace(workspace, lambda: linear_workspace_bytes(desc, "fwd"))
    check(lib().linear_fwd(C.byref(desc), *p, ws, nws, a.stream(stream)), "linear_fwd")
    return y


def linear_bwd(desc, dy, x, w, w_up=None, preact=None, offsets=None, dx=None, dw=None, dw_up=None, dbias=None,
               dbias_up=None, grad_accum=False, workspace=None, stream=None):
    """The gradients of :func:`linear_fwd` against ``dy`` [M, N], those asked for: ``dx`` [M, K], ``dw``
    (``dw_up``) like the weights, ``dbias`` (``dbias_up``). ``grad_accum``: the weight and bias gradients
    are fp32 buffers that are added to. The residual's gradient is ``dy``."""
    a = _Args()
    dt, _, ws_, bs, P = _linear_shapes(desc)
    gt = _F32 if grad_accum else dt
    M, K, N = desc.M, desc.K, desc.N
    p = (a(dy, "dy", dt, (M, N)), a(x, "x", dt, (M, K)), a(w, "w", dt, ws_), a.opt(w_up, "w_up", dt, ws_),
         a.opt(preact, "preact", dt, (M, P)), a.opt(offsets, "offsets", _I32, (desc.experts + 1,)),
         a.opt(dx, "dx", dt, (M, K)), a.opt(dw, "dw", gt, ws_), a.opt(dw_up, "dw_up", gt, ws_),
         a.opt(dbias, "dbias", gt, bs), a.opt(dbias_up, "dbias_up", gt, bs))
    keep, ws, nws = a.workspace(workspace, lambda: linear_workspace_bytes(desc, "bwd"))
    check(lib().linear_bwd(C.byref(desc), *p, int(bool(grad_accum)), ws, nws, a.stream(stream)), "linear_bwd")
