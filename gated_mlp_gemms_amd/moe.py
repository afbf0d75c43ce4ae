"""The mixture-of-experts operators of ``include/moe.h``: router, balance loss, tokens sorted by expert and back,
linear layer with its epilogue, experts' products, and their gradients.

As in the rest of the package the functions carry the C entry points' names, write into buffers the
caller passes, take a workspace (or allocate one with torch, on the stream that the call runs on) and run on
the current stream of their tensors' device unless ``stream`` is given. Sizes come from the tensors, so every tensor's dtype, shape
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

from . import _ACTS, _DTYPES
from ._lib import (LINEAR_ACT_NONE, LINEAR_BWD, LINEAR_FWD, MOE_SIGMOID, MOE_SOFTMAX, LinearDesc, MlpError, bind,
                   lib)

_SCORES = {"softmax": MOE_SOFTMAX, "sigmoid": MOE_SIGMOID}
_PHASES = {"fwd": LINEAR_FWD, "bwd": LINEAR_BWD}
_LINEAR_ACTS = {"none": LINEAR_ACT_NONE, **_ACTS}


def _score(score):
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    return code


# ---- router --------------------------------------------------------------------------------------

def moe_route(logits, ids, weights, score="softmax", renorm=True, stream=None):
    """The k largest of each token's E scores (``logits`` [T, E], f32 / bf16 / f16), largest first and
    ties to the lowest expert, into ``ids`` [T, k] (int32), and their probabilities into ``weights``
    [T, k] (fp32): ``score`` "softmax" over all experts or each one's "sigmoid", divided by the chosen
    ones' sum with ``renorm``. Scores of -inf are chosen last, with weight 0."""
    bind().moe_route(logits, ids, weights, _score(score), 1 if renorm else 0, stream)
    return ids, weights


def moe_route_bwd(logits, ids, dweights, dlogits, score="softmax", renorm=True, stream=None):
    """``dlogits`` [T, E] (logits' dtype): the gradient of :func:`moe_route`'s weights against
    ``dweights`` [T, k] (fp32), ``ids`` being what it chose."""
    bind().moe_route_bwd(logits, ids, dweights, dlogits, _score(score), 1 if renorm else 0, stream)
    return dlogits


# ---- balance loss ------------------------------------------------------------------------------------

def moe_balance_workspace_bytes(T, experts) -> int:
    b = lib().moe_balance_workspace_bytes(int(T), int(experts))
    if b == 0:
        raise MlpError(1, "moe_balance_workspace_bytes")
    return int(b)


def moe_balance(logits, ids, counts, shares, loss, mask=None, score="softmax", workspace=None, stream=None):
    """The load of each expert under the choices ``ids`` [T, k]: ``counts`` [E + 1] (int32, the last the number n
    of tokens that count), ``shares`` [E] (fp32) the mean probabilities (sigmoids divided by their sum), and
    ``loss`` [1] (fp32) = E sum_e counts[e] / (n k) shares[e]. ``mask`` [T] (bool): the tokens that count."""
    bind().moe_balance(logits, ids, mask, counts, shares, loss, _score(score), workspace, stream)
    return loss


def moe_balance_bwd(logits, ids, counts, dlogits, mask=None, dloss=None, dweights=None, score="softmax", renorm=True,
                    stream=None):
    """``dlogits`` [T, E]: ``dloss`` [1] (fp32, None: 1) times the gradient of :func:`moe_balance`'s loss, and with
    ``dweights`` [T, k] that of :func:`moe_route`'s weights added: the router's whole gradient, rounded once."""
    bind().moe_balance_bwd(logits, ids, mask, counts, dloss, dweights, dlogits, _score(score), 1 if renorm else 0, stream)
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
    bind().moe_sort(ids, experts, offsets, row_of, slot_of, workspace, stream)
    return offsets, row_of, slot_of


def moe_gather(x, slot_of, offsets, xs, stream=None):
    """``xs`` [T k, d]: row r is the row of ``x`` [T, d] that slot ``slot_of[r]`` belongs to; zeros
    behind ``offsets[E]``."""
    bind().moe_gather(x, slot_of, offsets, xs, stream)
    return xs


def moe_gather_bwd(dxs, row_of, offsets, dx, stream=None):
    """``dx`` [T, d]: each token's sum of its kept rows of ``dxs`` [T k, d], in fp32."""
    bind().moe_gather_bwd(dxs, row_of, offsets, dx, stream)
    return dx


def moe_combine(ys, weights, row_of, offsets, out, residual=None, stream=None):
    """``out`` [T, d] = ``residual`` + each token's kept rows of ``ys`` [T k, d] by ``weights`` [T, k]
    (fp32), summed in fp32 and rounded once. ``out`` may be ``residual``."""
    bind().moe_combine(ys, weights, row_of, offsets, out, residual, stream)
    return out


def moe_combine_bwd(dout, ys, weights, row_of, slot_of, offsets, dys, dweights, stream=None):
    """Both gradients of :func:`moe_combine` against ``dout`` [T, d]: ``dys`` [T k, d] (zeros in the
    dropped rows) and ``dweights`` [T, k] (fp32, 0 for a dropped slot). The residual's is ``dout``.
    It goes by rows and reads ``slot_of``; ``row_of``, its inverse, is only checked."""
    bind().moe_combine_bwd(dout, ys, weights, row_of, slot_of, offsets, dys, dweights, stream)
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


def linear_fwd(desc, x, w, y, w_up=None, bias=None, bias_up=None, residual=None, offsets=None, preact=None,
               workspace=None, stream=None):
    """``y`` [M, N] = residual + act(x w^T + bias), gated: act(x w^T + bias) (x w_up^T + bias_up).
    With experts, row r of ``x`` is of the expert e with offsets[e] <= r < offsets[e + 1]. ``preact``
    receives what the activation was taken of ([M, N], gated [M, 2N] = [g | u]), for linear_bwd."""
    bind().linear_fwd(desc, x, w, y, w_up, bias, bias_up, residual, offsets, preact, workspace, stream)
    return y


def linear_bwd(desc, dy, x, w, w_up=None, preact=None, offsets=None, dx=None, dw=None, dw_up=None, dbias=None,
               dbias_up=None, grad_accum=False, workspace=None, stream=None):
    """The gradients of :func:`linear_fwd` against ``dy`` [M, N], those asked for: ``dx`` [M, K], ``dw``
    (``dw_up``) like the weights, ``dbias`` (``dbias_up``). ``grad_accum``: the weight and bias gradients
    are fp32 buffers that are added to. The residual's gradient is ``dy``."""
    bind().linear_bwd(desc, dy, x, w, w_up, preact, offsets, dx, dw, dw_up, dbias, dbias_up, 1 if grad_accum else 0,
                      workspace, stream)
