"""The AdamW step and its 8-bit states, from the formulas, in fp64.

Test infrastructure only (see the package docstring).

    g = c grad, c = min(1, max_norm / (norm + 1e-6))
    m = b1 m + (1 - b1) g      v = b2 v + (1 - b2) g g
    p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)

8-bit states: OCP e4m3 (m) and e5m2 (v) with an fp32 scale per 256 elements, fl(a fl(1 / 448)) or
fl(a fl(1 / 57344)) for a block's largest magnitude a, 0 below 2^-100.  (The C call's definition: not the rounded
quotient, from which it is up to 2^-23 of itself away.)
"""
from __future__ import annotations

import numpy as np

__all__ = ["adamw_clip", "adamw_step", "state_codes", "state_values", "STATE_FORMATS"]

# (exponent bits, mantissa bits, bias, largest value)
STATE_FORMATS = {"m": (4, 3, 7, 448.0), "v": (5, 2, 15, 57344.0)}


def adamw_clip(grads, max_norm):
    norm = float(np.sqrt(sum(np.sum(np.square(g, dtype=np.float64)) for g in grads)))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def adamw_step(p, g, m, v, lr, beta1, beta2, eps, t, decay=0.0, clip=1.0):
    g = clip * g
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = p * (1 - lr * decay) - lr / (1 - beta1 ** t) * m / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p, m, v


def _levels(kind):
    """The non-negative values of a format, by code."""
    e, f, bias, top = STATE_FORMATS[kind]
    code = np.arange(1 << (e + f))
    exp, man = code >> f, code & ((1 << f) - 1)
    v = np.where(exp == 0, man * 2.0 ** (1 - bias - f), (1 + man / (1 << f)) * 2.0 ** (exp - bias))
    return v[v <= top]


def _blocks(x):
    x = np.asarray(x)
    return np.concatenate([x, np.zeros(-x.size % 256, x.dtype)]).reshape(-1, 256)


def state_codes(x, kind):
    """(codes, scales) of an fp32 vector."""
    n, x = x.size, _blocks(x.astype(np.float32))
    levels = _levels(kind)
    amax = np.abs(x).max(1)
    share = np.float32(1) / np.float32(STATE_FORMATS[kind][3])
    scale = np.where(amax < np.float32(2.0 ** -100), np.float32(0), amax * share).astype(np.float32)
    inverse = np.zeros_like(scale)
    np.divide(np.float32(1), scale, out=inverse, where=scale > 0)
    y = np.abs(x * inverse[:, None]).astype(np.float64)
    i = np.clip(np.searchsorted(levels, y), 1, levels.size - 1)
    lo, hi = y - levels[i - 1], levels[i] - y
    code = np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)   # ties to the even code
    if kind == "v":
        code = np.where((x > 0) & (scale[:, None] > 0) & (code == 0), 1, code)
    code = code + (np.signbit(x * inverse[:, None]) * (1 << sum(STATE_FORMATS[kind][:2])))
    return code.reshape(-1)[:n].astype(np.uint8), scale


def state_values(codes, scales, kind):
    e, f, _, _ = STATE_FORMATS[kind]
    half = 1 << (e + f)
    v = _levels(kind)[codes & (half - 1)] * np.where(codes >= half, -1.0, 1.0)
    return (v.astype(np.float32) * np.repeat(scales, 256)[:codes.size]).astype(np.float64)
