"""Training forward and gradient of an adapted layer, from their formulas, in fp64.

Test infrastructure only (see the package docstring).  W is the base weight's values
(bf16(deq) for NormalFloat, deq for MXFP4), A and B their bf16 roundings, keep the 0/1
mask of X or None, gain = alpha times the dropout scale.

    Y  = X W^T + gain (keep X) A^T B^T
    dX = G W + gain keep (G B A)      dB = gain G^T ((keep X) A^T)      dA = gain (G B)^T (keep X)
"""
from __future__ import annotations

import numpy as np

__all__ = ["layer_forward", "layer_backward"]


def _kept(M, keep):
    return M if keep is None else np.where(keep, M, 0.0)


def layer_forward(X, W, A, B, gain, keep=None, Xq=None):
    """Xq: what the base multiplies instead of X (MX(X) over an MXFP4 base)."""
    Y = (X if Xq is None else Xq) @ W.T
    return Y if A is None else Y + gain * (_kept(X, keep) @ A.T) @ B.T


def layer_backward(G, X, W, A, B, gain, keep=None):
    dX = G @ W
    if A is None:
        return dX, None, None
    Xd, P = _kept(X, keep), G @ B
    return dX + gain * _kept(P @ A, keep), gain * G.T @ (Xd @ A.T), gain * P.T @ Xd
