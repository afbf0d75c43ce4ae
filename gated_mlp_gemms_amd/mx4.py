"""Microscaled 4-bit floating point (``include/mx4.h``): blocks of 32 values with a power-of-two scale each, to
them, back, and the linear layer and the experts' products on them.

As in ``moe.py`` the functions carry the C entry points' names, write into buffers the caller passes, check every
tensor first (``ValueError``; what the library refuses raises ``MlpError``), take a workspace or allocate one, and
run on the current stream of their tensors' device unless ``stream`` is given. :func:`mx4_shapes` gives the shapes
of the two uint8 tensors that hold a matrix. A 4-bit layer, weights quantised once::

    mx4_quantize(w, wq, ws)                                  # [N, K], or [E, N, K]
    mx4_quantize(x, xq, xs)
    mx4_linear_fwd(desc, xq, xs, wq, ws, y)

and, of one weight without an activation, its backward's products, with the transposed blocks that ``mx4_quantize`` writes
next to the others (no bias' gradient; of experts ``dx`` only)::

    mx4_quantize(w, codes_t=wt, scales_t=wts)                # once: W^T, blocks along N
    mx4_quantize(x, codes_t=xt, scales_t=xts)
    mx4_quantize(dy, g, gs, codes_t=gt, scales_t=gts)
    mx4_linear_fwd(dx_desc, g, gs, wt, wts, dx)              # M x N -> K
    mx4_linear_fwd(dw_desc, gt, gts, xt, xts, dw)            # N rows of ceil(M / 32) 32 values -> K
"""
from __future__ import annotations

import ctypes as C

from ._lib import LinearDesc, MlpError, bind, lib


def mx4_shapes(rows, K, batch=None):
    """The shapes of the codes ([rows, K / 2]) and scales ([planes, scale rows, 8]) of a [rows, K] matrix, or of
    ``batch`` of them."""
    L, lead = lib(), () if batch is None else (int(batch),)
    return (*lead, int(rows), int(K) // 2), (*lead, int(L.mx4_planes(int(K))), int(L.mx4_scale_rows(int(rows))), 8)


def mx4_quantize(x, codes=None, scales=None, codes_t=None, scales_t=None, stream=None):
    """``x`` ([rows, cols] or [batch, rows, cols]) to 4-bit blocks along its rows (``codes``, ``scales``: shapes
    ``mx4_shapes(rows, cols)``), and / or of its transpose (``codes_t``, ``scales_t``: ``mx4_shapes(cols, deep)`` with deep
    the rows rounded up to a multiple of 32, zeros behind the last row)."""
    bind().mx4_quantize(x, codes, scales, codes_t, scales_t, stream)


def mx4_dequantize(codes, scales, out, stream=None):
    """``out`` ([rows, K] or [batch, rows, K]) = the values that codes and scales stand for, in its type."""
    bind().mx4_dequantize(codes, scales, out, stream)
    return out


def mx4_linear_workspace_bytes(desc: LinearDesc) -> int:
    n = lib().mx4_linear_workspace_bytes(C.byref(desc))
    if n == 0:
        raise MlpError(1, "mx4_linear_workspace_bytes")
    return int(n)


def mx4_linear_fwd(desc, x, x_scales, w, w_scales, y, w_up=None, w_up_scales=None, bias=None, bias_up=None,
                   residual=None, offsets=None, preact=None, workspace=None, stream=None):
    """:func:`linear_fwd` on 4-bit operands: ``y`` [M, N] = residual + act(x w^T + bias), gated: times
    (x w_up^T + bias_up); with experts, rows of ``x`` by ``offsets``. ``desc``'s dtype is that of y, bias,
    residual and preact. ``residual`` may be ``y``."""
    bind().mx4_linear_fwd(desc, x, x_scales, w, w_scales, y, w_up, w_up_scales, bias, bias_up, residual, offsets, preact,
                          workspace, stream)
    return y
