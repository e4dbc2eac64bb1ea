"""Buffers of codes with guarded surroundings, and inputs, for the tests of the operators on rows in 8 bits."""

from __future__ import annotations

import numpy as np
import torch

from tests.linear_util import Matrix, TORCH

FILL = 0x55


class CodeMatrix:
    """rows x cols int8 codes at a chosen row stride and offset (in codes) inside a buffer of one byte value."""

    dtype = "int8"

    def __init__(self, rows, cols, pad=0, offset=0, values=None):
        self.rows, self.cols, self.ld = rows, cols, cols + pad
        n = max(0, rows - 1) * self.ld + cols if rows and cols else 0
        self.start = 64 + offset
        self.buffer = torch.full((self.start + n + 64,), FILL, dtype=torch.int8, device="cuda")
        if values is not None:
            self.view.copy_(torch.as_tensor(values))
        self.snapshot()

    @property
    def view(self):
        return self.buffer.as_strided((self.rows, self.cols), (self.ld, 1), self.start)

    @property
    def ptr(self):
        return self.buffer.data_ptr() + self.start

    def snapshot(self):
        self.before = self.buffer.clone()

    def numpy(self):
        return self.view.cpu().numpy()

    def check_surroundings(self, what):
        now, want = self.buffer.clone(), self.before.clone()
        for t in (now, want):
            t.as_strided((self.rows, self.cols), (self.ld, 1), self.start).zero_()
        assert torch.equal(now, want), f"{what}: codes outside the matrix were written"


def vector(n, offset=0, values=None):
    """n floats at an odd place of a NaN-filled buffer."""
    return Matrix(1, n, "f32", offset=offset, values=None if values is None else np.asarray(values)[None, :])


def activations(seed, rows, cols, dtype):
    """Rows of different size with a few large channels, rounded to dtype, as a CPU tensor."""
    g = np.random.default_rng([seed, rows, cols])
    v = g.standard_normal((rows, cols)) * np.exp(0.5 * g.standard_normal((rows, 1)))
    v *= np.where(g.random(cols) < 0.02, 8.0, 1.0)
    return torch.from_numpy(v).to(TORCH[dtype])


def assert_codes(got, want, what):
    bad = got != want
    if bad.any():
        i = tuple(int(k[0]) for k in np.nonzero(bad))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} codes differ, first at {i}: got {got[i]}, want {want[i]}")
