"""The linear layer over block-scaled data and the gated activation, in float64 numpy.

Definitions only: a matrix of codes and scales becomes its float64 values (element value
times block scale, times the tensor scale for NV), and the products and the activation are
float64 from there. Shares nothing with the CUDA library.
"""

from __future__ import annotations

import numpy as np

import oracle

C = np.sqrt(2.0 / np.pi)


def table(fmt: str) -> np.ndarray:
    """float64 value of every code of a format (INT8: two's complement bytes)."""
    if fmt == "int8_sym":
        return np.arange(256, dtype=np.uint8).view(np.int8).astype(np.float64)
    n = 16 if fmt == "e2m1" else 256
    return np.array([oracle.fp_decode(fmt, c) for c in range(n)], dtype=np.float64)


def values(codes: np.ndarray, scales: np.ndarray, tensor_scale, rows: int, cols: int, scheme: oracle.Scheme) -> np.ndarray:
    """float64 [rows, cols] of MX or NV codes with row-major scales."""
    s = scheme.resolved()
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    if s.fmt == "e2m1":
        b = codes.reshape(rows, cols // 2)
        e = np.empty((rows, cols), dtype=np.uint8)
        e[:, 0::2], e[:, 1::2] = b & 15, b >> 4
    else:
        e = codes.reshape(rows, cols)
    v = table(s.fmt)[e]
    block = 32 if s.gran == "mx" else 16
    sc = np.ascontiguousarray(scales, dtype=np.uint8).reshape(rows, cols // block)
    f = np.ldexp(1.0, sc.astype(np.int32) - 127) if s.gran == "mx" else table("e4m3")[sc]
    v = v * np.repeat(f, block, axis=1)
    return v if s.gran == "mx" else v * float(np.asarray(tensor_scale).reshape(-1)[0])


def logistic(v: np.ndarray) -> np.ndarray:
    """1 / (1 + exp(-v)) without cancellation or overflow on either side."""
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def act(g: np.ndarray, kind: str):
    """a(g) = g s(v) and a'(g) = s + g s (1 - s) v' in float64 (1 - s(v) taken as s(-v))."""
    g = np.asarray(g, dtype=np.float64)
    if kind == "silu":
        v, dv = g, 1.0
    else:
        c = np.clip(g, -1e6, 1e6)      # beyond it s is 0 or 1; its cube overflows nothing
        v, dv = 2.0 * C * (c + 0.044715 * c ** 3), 2.0 * C * (1.0 + 3 * 0.044715 * c * c)
    s = logistic(v)
    return g * s, s + g * s * logistic(-v) * dv


def glu(g: np.ndarray, u: np.ndarray, kind: str) -> np.ndarray:
    return act(g, kind)[0] * np.asarray(u, dtype=np.float64)


def glu_backward(dh: np.ndarray, g: np.ndarray, u: np.ndarray, kind: str):
    """(dgate, dup) at the kept values g, u."""
    a, da = act(g, kind)
    dh = np.asarray(dh, dtype=np.float64)
    return dh * np.asarray(u, dtype=np.float64) * da, dh * a
