"""The dropout mask and dropout itself, from their definitions, in fp64.

Test infrastructure only (see the package docstring).

Element i of the row-major flattening is dropped where its 16 bits (lane i % 4, from the
low end, of output i // 4 of the SplitMix64 sequence started at the call's key) are below
thr = floor(2^16 p + 1/2), p as the fp32 number that the C call takes.  The key is output
``offset`` of the sequence started at ``seed``.  Kept elements are scaled by
2^16 / (2^16 - thr).
"""
from __future__ import annotations

import math

import numpy as np

from .rng import splitmix64_stream

__all__ = ["drop_threshold", "drop_scale", "keep_mask", "dropout"]


def drop_threshold(p: float) -> int:
    return int(math.floor(float(np.float32(p)) * 65536 + 0.5))


def drop_scale(p: float) -> float:
    thr = drop_threshold(p)
    return 0.0 if thr >= 65536 else 65536.0 / (65536 - thr)


def keep_mask(shape, p: float, seed: int, offset: int, first: int = 0) -> np.ndarray:
    """The kept elements of ``shape``, whose first element is element ``first`` of the call."""
    n = int(np.prod(shape))
    i = np.arange(first, first + n, dtype=np.uint64)
    key = int(splitmix64_stream(seed, np.array([offset % (1 << 64)], dtype=np.uint64))[0])
    word = splitmix64_stream(key, i >> np.uint64(2))
    bits = (word >> (np.uint64(16) * (i & np.uint64(3)))) & np.uint64(0xFFFF)
    return (bits >= np.uint64(drop_threshold(p))).reshape(shape)


def dropout(X: np.ndarray, p: float, seed: int, offset: int) -> np.ndarray:
    keep = keep_mask(X.shape, p, seed, offset)
    return np.where(keep, X.astype(np.float64) * drop_scale(p), 0.0)
