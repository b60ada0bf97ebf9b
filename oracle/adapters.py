"""Many adapters beside one shared weight, from the formulas, in fp64.

Test infrastructure only (see the package docstring).  A[s] (rank x cols) and B[s] (rows x rank)
are the slots' factors as they enter the products (bf16 roundings), slot_of[i] token i's slot (none
where it is not one of 0 .. slots - 1), ranks[s] a slot's own rank, gains[s] its whole factor
(alpha, the slot's gain and dropout's scale), keep the 0/1 mask of X or None.

    Y  = Y0 + gain (keep X) A^T B^T           each token with its own slot's factors
    dX = dX0 + gain keep (G B A)      dB = gain G^T ((keep X) A^T)      dA = gain (G B)^T (keep X)
"""
from __future__ import annotations

import numpy as np

__all__ = ["adapters_plan", "adapters_forward", "adapters_backward"]


def adapters_plan(slot_of, slots):
    """(starts, order): the tokens slot after slot, in rising order, those without an adapter last."""
    group = np.where((slot_of >= 0) & (slot_of < slots), slot_of, slots)
    order = np.concatenate([np.flatnonzero(group == s) for s in range(slots + 1)])
    return np.concatenate([[0], np.cumsum(np.bincount(group, minlength=slots + 1))]), order


def _slots(slot_of, B, ranks):
    for s in range(B.shape[0]):
        at = np.flatnonzero(slot_of == s)
        r = B.shape[2] if ranks is None else int(np.clip(ranks[s], 0, B.shape[2]))
        if at.size and r:
            yield s, at, r


def adapters_forward(X, B, A, slot_of, gains, ranks=None, keep=None, Y0=None):
    Y = np.zeros((X.shape[0], B.shape[1])) if Y0 is None else Y0.astype(np.float64)
    Xd = X if keep is None else np.where(keep, X, 0.0)
    for s, at, r in _slots(slot_of, B, ranks):
        Y[at] += gains[s] * (Xd[at] @ A[s, :r].T) @ B[s, :, :r].T
    return Y


def adapters_backward(G, X, B, A, slot_of, gains, ranks=None, keep=None, dX0=None):
    dX = np.zeros(X.shape) if dX0 is None else dX0.astype(np.float64)
    dB, dA = np.zeros(B.shape), np.zeros(A.shape)
    Xd = X if keep is None else np.where(keep, X, 0.0)
    for s, at, r in _slots(slot_of, B, ranks):
        P = G[at] @ B[s, :, :r]
        term = gains[s] * P @ A[s, :r]
        dX[at] += term if keep is None else np.where(keep[at], term, 0.0)
        dB[s, :, :r] = gains[s] * G[at].T @ (Xd[at] @ A[s, :r].T)
        dA[s, :r] = gains[s] * P.T @ Xd[at]
    return dX, dB, dA
