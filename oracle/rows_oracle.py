"""Rows in 8 bits, the root-mean-square norm with its gradients, and products of 8-bit rows, from their definitions.

numpy in float64 (integers for the products of codes); shares no code with the library.  Matrices are float64 arrays
of the values that their elements hold.
"""

from __future__ import annotations

import numpy as np


def quantize_oracle(v):
    """(codes, scales) of each row: the whole number nearest to 127 v / max|v|, ties to even, and max|v| / 127.

    v's elements have at most 35 significant bits, so that 127 |v| and the remainders here are exact.
    """
    v = np.asarray(v, dtype=np.float64)
    top = np.abs(v).max(1, initial=0.0) if v.shape[1] else np.zeros(v.shape[0])
    bad = ~np.isfinite(v).all(1)
    unit = np.where(bad | (top == 0), 1.0, top)[:, None]
    size = np.where(bad[:, None], 0.0, np.abs(v)) * 127.0
    whole = np.floor(size / unit)
    twice = 2.0 * (size - whole * unit)
    up = (twice > unit) | ((twice == unit) & (whole % 2 == 1))
    codes = np.where(bad[:, None], 0.0, np.sign(v) * (whole + up))
    return codes.astype(np.int8), np.where(bad, np.nan, top / 127.0)


def norm_oracle(h, weight, eps):
    """(y, rstd, codes, scales) of rows h that hold the rounded sums already."""
    mean = (h * h).sum(1) / max(h.shape[1], 1)
    rstd = 1.0 / np.sqrt(mean + eps)
    v = h if weight is None else h * weight
    codes, scales = quantize_oracle(v)
    return v * rstd[:, None], rstd, codes, scales * rstd


def norm_backward_oracle(dy, h, rstd, weight=None, dh=None):
    """(dx, dw) for the gradients dy of y and dh of h."""
    n = h * rstd[:, None]
    g = dy if weight is None else dy * weight
    dx = rstd[:, None] * (g - n * ((g * n).sum(1) / max(h.shape[1], 1))[:, None])
    return (dx if dh is None else dx + dh), (dy * n).sum(0)


def codes_product_oracle(x, w, x_scale, w_scale):
    """x_scale[m] w_scale[n] sum_k x(m,k) w(n,k) of int8 codes; the sums are exact."""
    total = x.astype(np.float64) @ w.astype(np.float64).T       # below 2^53
    return total * x_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)[None, :]
