"""Buffers with guarded surroundings for the linear layer's and AdamW's tests, and their error bounds."""

from __future__ import annotations

import numpy as np
import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# a rounding to nearest is off by at most half a step: finfo.eps / 2 relative to the value
HALF_STEP = {t: torch.finfo(d).eps / 2 for t, d in TORCH.items()}
# and by at most half of the smallest subnormal, for values below the normal ones
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}
U32 = 2.0 ** -24
# activations and slopes are evaluated in fp32 by a few operations of about one ulp each
ACT_ERROR = 2.0 ** -19


# M, N, K of the larger products.  Between them they reach every tile in every layout, whole and cut.
LARGE = [(33, 600, 4100), (130, 520, 3000), (1000, 1030, 2050), (1100, 2300, 200), (2048, 1024, 512), (700, 700, 8192),
         (2100, 2300, 520), (600, 1100, 8300), (8300, 1100, 600), (1100, 8300, 600)]
HUGE = [(4352, 4000, 4096), (4000, 4352, 4100), (4608, 4096, 1200)]


class Matrix:
    """rows x cols elements at a chosen row stride and offset inside a buffer filled with NaN."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0, values=None, device="cuda"):
        self.rows, self.cols, self.ld, self.dtype = rows, cols, cols + pad, dtype
        n = max(0, rows - 1) * self.ld + cols if rows and cols else 0
        self.start = 64 + offset
        self.buffer = torch.full((self.start + n + 64,), float("nan"), dtype=TORCH[dtype], device=device)
        self.before = None
        if values is not None:
            self.view.copy_(torch.as_tensor(values))
        self.snapshot()

    @property
    def view(self):
        return self.buffer.as_strided((self.rows, self.cols), (self.ld, 1), self.start)

    @property
    def ptr(self):
        return self.buffer.data_ptr() + self.start * self.buffer.element_size()

    def snapshot(self):
        bits = torch.int32 if self.dtype == "f32" else torch.int16
        self.before = self.buffer.view(bits).clone()

    def f64(self) -> np.ndarray:
        return self.view.double().cpu().numpy()

    def check_surroundings(self, what):
        """Nothing outside the matrix has changed since the snapshot."""
        bits = self.before.dtype
        now, want = self.buffer.view(bits).clone(), self.before.clone()
        for t in (now, want):
            t.as_strided((self.rows, self.cols), (self.ld, 1), self.start).zero_()
        assert torch.equal(now, want), f"{what}: elements outside the matrix were written"


def random_matrix(seed, rows, cols, dtype, scale=1.0, **kw) -> Matrix:
    g = np.random.default_rng([seed, rows, cols])
    return Matrix(rows, cols, dtype, values=torch.from_numpy(g.standard_normal((rows, cols)) * scale).to(TORCH[dtype]), **kw)


def assert_close(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err - bound)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} elements past their bound, worst at {i}: "
                             f"got {got[i]!r}, want {want[i]!r}, bound {bound[i]!r}")


def product_bound(a, b, terms):
    """How far an fp32 accumulation of a b^T (float64 arrays of exact operands) may be off."""
    return (terms + 8) * U32 * (np.abs(a) @ np.abs(b).T)


def rounded_bound(want, before, dtype):
    """Bound after one rounding to dtype of a value that is `before` off."""
    h = HALF_STEP[dtype]
    return before * (1 + h) + h * np.abs(want) + TINY[dtype]
