"""Weight gradients from x kept in 8 bits in fp16, for gradients and scales far from 1, against the float64 oracle.

dz times a rest of its row's scale is held in fp16 beside the codes times a power of two 2^b, where scale = rest 2^b, and b is chosen
from the scale and the row's largest finite |dy|, D.  So an element of dz is off by half an fp16 step (h = 2^-11) of itself, or of

    L = max(2^-13 D, 2^-38 / scale)

where it is smaller: D rest is at least 1/2 unless b is -24 already, and fp16's smallest normal number is 2^-14, which is 2^-13 of
1/2 and a dz of 2^-38 / scale.  A second term, for dw in fp32, is off by half a step of what the first leaves, or of L.

The matrix instruction's fp32 sums are off by 2^-24 of their terms' magnitudes for each addition, but a subnormal factor q 2^b counts
as 2^-14 there (its product is added without being normalised), as if x were scale 2^(-14-b): measured for q up to 127 and up to 3
and b from 0 to -24, where the errors grow with max(|q| 2^b, 2^-14).
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import linear_backward_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import ACT_ERROR, HALF_STEP, U32, assert_close, rounded_bound
from tests.test_linear_backward_q8_gpu import BackwardQ8

pytestmark = pytest.mark.gpu

H = HALF_STEP["f16"]


class Small(BackwardQ8):
    """Gradients of fp16 rows, dy of about `size`; x is `x_size` times what it was."""

    def __init__(self, M, N, K, size, act="none", dw_dtype="f32", x_size=1.0, **kw):
        super().__init__(M, N, K, "f16", act, dw_dtype, **kw)
        self.dy.view.mul_(size)
        self.dy.snapshot()
        self.x.scale.view.mul_(x_size)
        self.x.scale.snapshot()

    def weight_gradient(self):
        """(dw, bound)"""
        M = self.shape[0]
        dy, x = self.dy.f64(), self.x.f64()
        z = self.z.f64() if self.z else np.zeros_like(dy)
        _, dw, _, dz = linear_backward_oracle(dy, z, x, self.w.f64(), self.act)
        dz_off = (ACT_ERROR * (1 + np.abs(z)) + U32 + 1.2 * U32 * np.abs(z)) * np.abs(dy) if self.act != "none" else np.zeros_like(dy)
        top = np.where(np.isfinite(dy), np.abs(dy), 0.0).max(1, keepdims=True)
        scale = np.abs(self.x.scale.f64().T)
        least = np.maximum(2.0 ** -13 * top, 2.0 ** -38 / np.where(scale > 0, scale, np.inf))
        e = np.frexp(scale)[1] + np.maximum(np.frexp(np.where(top > 0, top, 2.0 ** -24))[1], -23) - 15
        b = np.where(e >= -18, np.minimum(e, 8), np.maximum(np.minimum(e + 14, -18), -24))
        counts = np.maximum(np.abs(x), scale * 2.0 ** (-14 - b))
        folded = dz_off + U32 * np.abs(dz)
        left = H * np.maximum(np.abs(dz) + folded, least)
        if self.dw_dtype == "f32":
            left = H * np.maximum(left, least)
        dz_w = folded + left
        sums = (2 if self.dw_dtype == "f32" else 1) * (M + 10)
        off = dz_w.T @ np.abs(x) + sums * U32 * ((np.abs(dz) + dz_w).T @ counts)
        if self.accumulate:
            dw = dw + self.dw0
            off = off + 2 * U32 * (np.abs(dw) + np.abs(self.dw0))
        return dw, rounded_bound(dw, off, self.dw_dtype)

    def check_weight_gradient(self, what):
        torch.cuda.synchronize()
        want, bound = self.weight_gradient()
        assert_close(self.dw.f64(), want, bound, what)
        self.dw.check_surroundings(what)


# rows of 16, 64 and 256 threads; dz's terms in one product and, past 32 rows for a column, in a product each
SHAPES = [(6, 40, 24), (40, 24, 16), (300, 8, 40), (5, 300, 1000), (70, 2100, 300), (7, 30, 4100), (1, 5000, 2500), (2, 9000, 70)]


@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_small_gradients_in_fp32(M, N, K, size):
    require_gpu()
    for act, acc in (("none", False), ("gelu", False), ("none", True)):
        what = f"dw f32 {M}x{N}x{K} {act} dy {size} accumulate {acc}"
        log(what)
        b = Small(M, N, K, size, act, accumulate=acc, pad=3 if acc else 0, z8=not acc)
        if acc:
            b.dw.view.mul_(size)
            b.dw0 = b.dw.f64()
            b.dw.snapshot()
        b.run()
        b.check_weight_gradient(what)


@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_small_gradients_in_fp16(M, N, K, size):
    """x of about 64, so that dw is well inside fp16."""
    require_gpu()
    for act in ("none", "relu"):
        what = f"dw f16 {M}x{N}x{K} {act} dy {size}"
        log(what)
        b = Small(M, N, K, size, act, "f16", x_size=64.0)
        b.run()
        b.check_weight_gradient(what)


@pytest.mark.parametrize("exponent", [-40, -30, -27, -25, -24, -12, 0, 8, 12])
def test_scales_from_tiny_to_large(exponent):
    require_gpu()
    for size in (1.0, 1e-3):
        what = f"dw f32, scales 1.5 x 2^{exponent}, dy {size}"
        log(what)
        b = Small(40, 24, 16, size)
        b.x.scale.view.fill_(1.5 * 2.0 ** exponent)
        b.x.scale.snapshot()
        b.run()
        b.check_weight_gradient(what)


def test_rows_of_different_size():
    """Each row's power of two is its own: rows from 2^-20 to 2^15 of dy beside scales from 2^-18 to 2^6, and a row of zeros."""
    require_gpu()
    for M, N, K in ((36, 40, 24), (36, 520, 1000), (36, 4100, 136)):
        log(f"dw f32 {M}x{N}x{K} of rows of different size")
        b = Small(M, N, K, 1.0)
        b.dy.view.clamp_(-1, 1)
        b.dy.view.mul_(torch.exp2(torch.arange(-20, 16, device="cuda").float())[:, None])
        b.dy.view[7] = 0.0
        b.dy.snapshot()
        b.x.scale.view.copy_(1.25 * torch.exp2(6 - torch.arange(36, device="cuda").float() * 24 / 35)[None])
        b.x.scale.snapshot()
        b.run(dx=None, w=None)
        b.check_weight_gradient("rows of different size")


def test_infinities_and_nan_in_dy():
    """They reach their own column of dz, a row of dw; the row's other elements are as exact as without them."""
    require_gpu()
    for M, N, K in ((12, 40, 24), (12, 600, 24), (12, 40, 2100)):
        log(f"dw f32 {M}x{N}x{K} with an infinity and a NaN in dy")
        b = Small(M, N, K, 1e-5)
        b.dy.view[3, 5], b.dy.view[4, 6], b.dy.view[5, N - 1] = float("inf"), float("nan"), float("-inf")
        b.dy.snapshot()
        b.run(dx=None, w=None, db=None)
        torch.cuda.synchronize()
        got = b.dw.f64()
        poisoned = [5, 6, N - 1]
        assert not np.isfinite(got[poisoned]).any()
        others = np.delete(np.arange(N), poisoned)
        with np.errstate(invalid="ignore"):
            want, bound = b.weight_gradient()
        assert_close(got[others], want[others], bound[others], "the other columns of dz")


def test_zero_and_nan_scales():
    require_gpu()
    for dw in ("f32", "f16"):
        log(f"dw {dw} with a zero scale, then a NaN")
        b = Small(20, 40, 24, 1e-3, dw_dtype=dw)
        b.x.codes.view[4] = 0
        b.x.scale.view[0, 4] = 0.0
        b.run()
        b.check_weight_gradient("a scale of 0")
        b.x.scale.view[0, 4] = float("nan")
        b.run()
        torch.cuda.synchronize()
        assert np.isnan(b.dw.f64()).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(159, 4, 264), (160, 4, 264), (8300, 300, 8200)])
def test_both_sides_of_the_copies_limits(M, N, K, dtype):
    """dw in fp32 with a copy of x per term, and past 32 rows for a column or 128 MiB of copies with a product per term."""
    require_gpu()
    for acc in (False, True) if M < 1000 else (True,):
        what = f"linear_backward_q8 {M}x{N}x{K} {dtype} dw f32 accumulate {acc}"
        log(what)
        b = BackwardQ8(M, N, K, dtype, "gelu", "f32", acc, seed=M)
        b.run()
        b.check(what)


@pytest.mark.parametrize("dw_dtype", ["f16", "f32"])
def test_in_a_graph(dw_dtype):
    """Captured once, replayed on gradients of other sizes, with eager calls on another workspace between: the powers are each replay's."""
    require_gpu()
    log(f"linear_backward_q8 f16 dw {dw_dtype} in a graph")
    b = Small(70, 520, 264, 1.0, "gelu", dw_dtype)
    a = b.args()
    need = ag.plan_linear_backward_q8(**a).workspace_bytes
    space, other = (torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ag.linear_backward_q8(**a, workspace=space, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ag.linear_backward_q8(**a, workspace=space, stream=side)
    g = torch.Generator(device="cuda").manual_seed(1)
    for size in (1.0, 1e-4, 1e3, 1e-6):
        b.dy.view.copy_(torch.randn(b.dy.view.shape, generator=g, device="cuda") * size)
        b.dy.snapshot()
        graph.replay()
        torch.cuda.synchronize()
        got = [m.buffer.clone() for m in (b.dx, b.dw, b.db)]
        ag.linear_backward_q8(**a, workspace=other)
        torch.cuda.synchronize()
        same = lambda u, v: torch.equal(u.view(torch.uint8), v.view(torch.uint8))  # noqa: E731
        assert all(same(u, m.buffer) for u, m in zip(got, (b.dx, b.dw, b.db))), f"replay at {size}"
        b.check_weight_gradient(f"replay at {size}")
