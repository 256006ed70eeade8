"""Oracle of the packed-MXFP4 operators -- test infrastructure.

Plain NumPy in 64 bits, from the definitions: blocks of 32 along a row share
2^e, e = floor(log2 m) - 2 with m the block's largest magnitude (at least
-127; 0 for a block of zeros), elements are the E2M1 values nearest x / 2^e
(float_formats.e2m1_round), a block without a finite fp32 maximum has scale
byte 255 and zero codes and stands for NaN.  Two codes a byte, the even column
in the low nibble.
"""
from __future__ import annotations

import numpy as np

from .float_formats import e2m1_round, e2m1_table

F32, F64 = np.float32, np.float64


def quantize(x, alpha=None):
    """(codes [M, K], scale bytes [M, K/32]) of x, fp64 (or exact in it)."""
    x = np.asarray(x, F64)
    m, k = x.shape
    b = x.reshape(m, k // 32, 32)
    with np.errstate(over="ignore", invalid="ignore"):
        top = np.abs(b).max(axis=2)
        if alpha is not None:      # the clip is an fp32 product
            top = np.abs(np.asarray(alpha, F32) * top.astype(F32)).astype(F64)
        top32 = top.astype(F32)
    fine = np.isfinite(top32)
    some = fine & (top32 > 0)
    e = np.zeros(top.shape, np.int64)
    e[some] = np.maximum(np.frexp(top[some])[1] - 1 - 2, -127)     # frexp: top = f 2^n, f in [1/2, 1)
    y = np.where(fine[..., None], b, 0.0) * np.ldexp(1.0, -e)[..., None]
    _, codes = e2m1_round(y)
    scale = np.where(fine, e + 127, 255).astype(np.uint8)
    return np.where(fine[..., None], codes, 0).astype(np.uint8).reshape(m, k), scale


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def values(packed, scale):
    """fp64 values [M, K] of packed codes and scale bytes."""
    mags = e2m1_table()[1]
    table = np.concatenate([mags, -mags])
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    v = table[unpack(packed)]
    return (v.reshape(*scale.shape, 32) * s[..., None]).reshape(v.shape)


def residual(x, delta, c):
    """x + c delta in fp32, each operation rounded."""
    x = np.asarray(x, F32)
    return x if delta is None else (x + (F32(c) * np.asarray(delta, F32)).astype(F32)).astype(F32)


def rmsnorm(r, w, eps):
    r = np.asarray(r, F64)
    with np.errstate(invalid="ignore", divide="ignore"):
        h = r / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + F64(F32(eps)))
        return h if w is None else h * np.asarray(w, F64)


def swiglu(g, u):
    g, u = np.asarray(g, F64), np.asarray(u, F64)
    with np.errstate(over="ignore", invalid="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def product(x, w):
    """(X W^T, |X| |W|^T) in fp64."""
    return np.asarray(x, F64) @ np.asarray(w, F64).T, np.abs(x) @ np.abs(w).T
