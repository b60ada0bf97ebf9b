"""MXFP4 (OCP Microscaling Formats v1.0) quantization, written out plainly.

Test infrastructure only (see the package docstring).

Blocks are 32 consecutive columns of a row; the row's last block may be shorter.  The scale
is 2^(byte - 127) with byte = max(0, floor(log2 amax) - 2 + 127) (2 is the exponent of FP4's
largest binade), 0 for a zero block and 255 (NaN) for one that holds an infinity or a NaN.
Elements are rounded to the nearest of the e2m1 values, a tie to the even code, larger
magnitudes to 6.
"""
from __future__ import annotations

import numpy as np

__all__ = ["E2M1", "mx_scale_bytes", "mx_quantize", "mx_values", "mx_pack", "mx_unpack"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _blocks(R: np.ndarray) -> np.ndarray:
    rows, cols = R.shape
    steps = -(-cols // 256)
    out = np.zeros((rows, steps * 256), dtype=np.float64)
    out[:, :cols] = R
    return out.reshape(rows, steps * 8, 32)


def mx_scale_bytes(R: np.ndarray) -> np.ndarray:
    """rows x (whole steps of 8) scale bytes."""
    amax = np.abs(_blocks(R)).max(2)
    fine = np.isfinite(amax)
    exponent = np.frexp(np.where(fine & (amax > 0), amax, 1.0))[1] - 1
    byte = np.where(amax > 0, np.maximum(0, exponent - 2 + 127), 0)
    return np.where(fine, byte, 255).astype(np.uint8)


def mx_quantize(R: np.ndarray):
    """(codes rows x padded cols, scale bytes rows x blocks) of an fp32 matrix."""
    b = _blocks(R)
    byte = mx_scale_bytes(R)
    with np.errstate(invalid="ignore"):
        x = b / np.exp2(byte.astype(np.float64) - 127)[:, :, None]
        x[byte == 255] = 0.0
    # how many midpoints of neighbours lie below; one that is met counts where the code above it is even
    m, mids = np.abs(x), 0.5 * (E2M1[1:] + E2M1[:-1])
    pick = sum(((m >= v) if (k + 1) % 2 == 0 else (m > v)).astype(np.uint8) for k, v in enumerate(mids))
    codes = (pick + 8 * np.signbit(x)).astype(np.uint8)
    return codes.reshape(R.shape[0], -1), byte


def mx_values(codes: np.ndarray, byte: np.ndarray, cols: int) -> np.ndarray:
    scale = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    sign = np.where(codes & 8, -1.0, 1.0)
    v = sign * E2M1[codes & 7]
    return (v.reshape(byte.shape + (32,)) * scale[:, :, None]).reshape(codes.shape)[:, :cols]


def mx_pack(codes: np.ndarray, byte: np.ndarray):
    """The library's storage: two codes per byte, the first in the high nibble; scales by steps of 8."""
    rows = codes.shape[0]
    packed = (codes[:, 0::2] << 4 | codes[:, 1::2]).astype(np.uint8)
    return packed, np.ascontiguousarray(byte.reshape(rows, -1, 8).transpose(1, 0, 2))


def mx_unpack(packed: np.ndarray, scales: np.ndarray):
    codes = np.stack((packed >> 4, packed & 15), -1).reshape(packed.shape[0], -1)
    return codes, np.ascontiguousarray(scales.transpose(1, 0, 2)).reshape(packed.shape[0], -1)
