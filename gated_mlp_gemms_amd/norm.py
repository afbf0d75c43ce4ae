"""The norm in front of a layer (``include/norm.h``): layer norm or RMS norm of the residual stream, with the
sum of what the layer before added, and the gradients.

As in ``moe.py`` the functions carry the C entry points' names, write into buffers the caller passes, check every
tensor first (``ValueError``; what the library refuses raises ``MlpError``), take a workspace or allocate one, and
run on the current stream of their tensors' device unless ``stream`` is given. A pre-norm layer::

    norm_fwd(x, y, weight=w, bias=b, residual=r, h=h, mean=mean, rstd=rstd)   # h = x + r, y = norm(h) w + b
    ...                                                                       # y -> out, added onto h
    norm_bwd(dy, h, rstd, dh, mean=mean, weight=w, dresidual=dout, dweight=dw, dbias=db)

``dh`` is the gradient of ``x`` and of ``residual`` alike.
"""
from __future__ import annotations

from ._lib import NORM_LAYER, NORM_RMS, MlpError, bind, lib

_KINDS = {"layer": NORM_LAYER, "rms": NORM_RMS}


def _kind(kind):
    code = _KINDS.get(kind)
    if code is None:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}, not {kind!r}")
    return code


def norm_fwd(x, y, weight=None, bias=None, residual=None, h=None, mean=None, rstd=None, kind="layer", eps=1e-5,
             stream=None):
    """``y`` [M, d] = the norm of ``x`` (+ ``residual``) times ``weight`` plus ``bias`` ([d], of x's type or
    fp32). With a residual ``h`` receives the sum, rounded, which the norm is taken of (it may be ``x`` or
    ``residual``); ``mean`` (layer norm) and ``rstd`` [M] (fp32) receive the statistics for :func:`norm_bwd`."""
    bind().norm_fwd(x, y, weight, bias, residual, h, mean, rstd, _kind(kind), eps, stream)
    return y


def norm_workspace_bytes(M, d) -> int:
    b = lib().norm_workspace_bytes(int(M), int(d))
    if b == 0:
        raise MlpError(1, "norm_workspace_bytes")
    return int(b)


def norm_bwd(dy, h, rstd, dx=None, mean=None, weight=None, dresidual=None, dweight=None, dbias=None, kind="layer",
             grad_accum=False, workspace=None, stream=None):
    """The gradients of :func:`norm_fwd` against ``dy`` [M, d], those asked for: ``dx`` [M, d], of h, with
    ``dresidual`` added (``dx`` may be it); ``dweight``, ``dbias`` [d] in the weights' type, or added into fp32
    buffers with ``grad_accum``. ``mean`` belongs to layer norm only."""
    bind().norm_bwd(dy, h, mean, rstd, weight, dresidual, dx, dweight, dbias, _kind(kind), 1 if grad_accum else 0,
                    workspace, stream)
