"""64-bit definitions of the MXFP4 block, its products and the norms around a block of a model.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

An MXFP4 tensor [rows][cols] is a plane of 4-bit codes (low nibble first), then one byte p for every 32 columns:
w = 2^(p - 127) * value(code), p = 255 NaN.  A code is a float of one sign bit, two exponent bits (bias 1) and one
mantissa bit, written from that definition here."""
from __future__ import annotations

import numpy as np

from .gemv import silu64


def code_values() -> np.ndarray:
    """The sixteen values: (-1)^s * m / 2 for e = 0, (-1)^s * (1 + m / 2) * 2^(e - 1) else."""
    out = np.zeros(16)
    for c in range(16):
        s, e, m = c >> 3, (c >> 1) & 3, c & 1
        v = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        out[c] = -v if s else v
    return out


def mx4_pack(p: np.ndarray, code: np.ndarray) -> np.ndarray:
    code = np.asarray(code, np.uint8)
    return np.concatenate([(code[:, 0::2] | (code[:, 1::2] << 4)).reshape(-1), np.asarray(p, np.uint8).reshape(-1)])


def mx4_unpack(data: np.ndarray, rows: int, cols: int):
    b = data[:rows * cols // 2].reshape(rows, cols // 2)
    return data[rows * cols // 2:].reshape(rows, cols // 32), np.stack([b & 15, b >> 4], -1).reshape(rows, cols)


def mx4_decode64(data: np.ndarray, rows: int, cols: int) -> np.ndarray:
    p, code = mx4_unpack(np.asarray(data, np.uint8), rows, cols)
    scale = np.where(p == 255, np.nan, np.ldexp(1.0, p.astype(np.int64) - 127))
    return code_values()[code] * np.repeat(scale, 32, axis=1)


def mx4_encode64(x: np.ndarray):
    """(p, code) of rows x (float64 holding the given numbers exactly): the power that brings a block's largest into
    [4, 8), at least 2^-127; the nearest value, of two as near the even code; a block with NaN or infinity: p = 255,
    codes 0."""
    rows, cols = x.shape
    b = np.asarray(x, np.float64).reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    _, e = np.frexp(top)  # top in [2^(e - 1), 2^e)
    p = np.where(top > 0, np.maximum(0, e - 1 - 2 + 127), 0)
    mag = np.abs(np.ldexp(b, 127 - p[..., None]))
    vals = code_values()[:8]
    d = np.abs(mag[..., None] - vals)
    near = d.min(-1)
    code = np.zeros(b.shape, np.int64)
    for c in list(range(1, 8, 2)) + list(range(0, 8, 2)):  # even codes last: they win ties
        code = np.where(d[..., c] == near, c, code)
    code = code | (np.signbit(b) * 8)
    code = np.where(bad[..., None], 0, code)
    return np.where(bad, 255, p).astype(np.uint8), code.reshape(rows, cols).astype(np.uint8)


def swiglu_halves(y: np.ndarray) -> np.ndarray:
    n = y.shape[1] // 2
    return silu64(y[:, :n]) * y[:, n:]


def groups(expert_start, rows: int):
    """(first, end) of every expert: the running maximum of its numbers, cut to [0, rows]."""
    s = np.maximum.accumulate(np.clip(np.asarray(expert_start, np.int64), 0, rows))
    return list(zip(s[:-1], s[1:]))


def norm64(x: np.ndarray, kind, weight=None, bias=None, eps: float = 1e-6) -> np.ndarray:
    if kind is None:
        return x
    x = x - x.mean(-1, keepdims=True) if kind == "layer" else x
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = y if weight is None else y * weight
    return y if bias is None else y + bias
