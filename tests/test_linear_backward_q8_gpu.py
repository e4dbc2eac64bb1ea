"""The linear layer's gradients from activations kept in 8 bits, on the GPU against the float64 oracle of the kept values.

The bounds are those of the gradients without codes, with what the codes add: dw's dz is multiplied by a factor of its
row's scale (one fp32 rounding) before its rounding to 16 bits, and a kept z is an fp32 product (one rounding, through a slope
that changes by at most 1.2 for a step of one).  The codes' own products with the scale's power of two are exact.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import linear_backward_oracle
from oracle.rows_oracle import quantize_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import ACT_ERROR, HALF_STEP, HUGE, LARGE, TINY, U32, assert_close, rounded_bound
from tests.rows_util import CodeMatrix, vector
from tests.test_linear_gpu import ACTS, SIZES, Backward, workspace

pytestmark = pytest.mark.gpu


class Kept:
    """A matrix as its codes and scales stand for it."""

    def __init__(self, m, pad, offset):
        codes, scales = quantize_oracle(m.f64())
        self.codes = CodeMatrix(m.rows, m.cols, pad, offset, codes)
        self.scale = vector(m.rows, offset, scales.astype(np.float32))
        self.ptr, self.ld = self.codes.ptr, self.codes.ld

    def f64(self):
        return self.codes.numpy().astype(np.float64) * self.scale.f64().T


class BackwardQ8(Backward):
    def __init__(self, M, N, K, dtype, act="none", dw_dtype=None, accumulate=False, db=True, pad=0, offset=0, seed=1, x8=True, z8=True):
        super().__init__(M, N, K, dtype, act, dw_dtype, accumulate, db, pad, offset, seed)
        self.x8, self.z8 = x8, z8 and act != "none"
        self.terms = 3 if x8 and dtype == "bf16" else 2         # of dz for a dw in fp32
        if x8:
            self.x = Kept(self.x, pad, offset)
        if self.z8:
            self.z = Kept(self.z, pad, offset)

    def args(self):
        return dict(super().args(), x_scale=self.x.scale.ptr if self.x8 else None, z_scale=self.z.scale.ptr if self.z8 else None)

    def run(self, stream=None, **over):
        a = dict(self.args(), **over)
        ag.linear_backward_q8(**a, workspace=workspace(ag.plan_linear_backward_q8(**a)), stream=stream)

    def bounds(self):
        M, N, K = self.shape
        dy, x, w = self.dy.f64(), self.x.f64(), self.w.f64()
        z = self.z.f64() if self.z else np.zeros_like(dy)
        dx, dw, db, dz = linear_backward_oracle(dy, z, x, w, self.act)
        # relu's slope has no error; a kept z that is not zero keeps its sign
        dz_off = (ACT_ERROR * (1 + np.abs(z)) + U32 + 1.2 * U32 * np.abs(z)) * np.abs(dy) if self.act != "none" else np.zeros_like(dy)
        dz_x = rounded_bound(dz, dz_off, self.dtype) if self.act != "none" else dz_off
        h, tiny = HALF_STEP[self.dtype], TINY[self.dtype]
        folded = dz_off + U32 * np.abs(dz)
        if not self.x8:
            dz_w = dz_x if self.dw_dtype != "f32" or self.act == "none" else dz_off + h * (h * (np.abs(dz) + dz_off) + tiny) + tiny
        elif self.dw_dtype == "f32":        # each term is what the one before leaves, half a step of it
            dz_w = h * (np.abs(dz) + folded) + 2 * tiny
            for _ in range(self.terms - 1):
                dz_w = h * dz_w + 2 * tiny
            dz_w = folded + dz_w
        else:                               # the factor is at least 1/2
            dz_w = folded + h * (np.abs(dz) + folded) + 2 * tiny
        size, size_w = np.abs(dz) + dz_x, np.abs(dz) + dz_w
        off_x = dz_x @ np.abs(w) + (N + 8) * U32 * (size @ np.abs(w))
        sums = self.terms * (M + 10) if self.dw_dtype == "f32" else M + 8
        off_w = dz_w.T @ np.abs(x) + sums * U32 * (size_w.T @ np.abs(x))
        off_b = dz_off.sum(0) + (M + 8) * U32 * size.sum(0)
        if self.accumulate:
            dw = dw + self.dw0
            off_w = off_w + self.terms * U32 * (np.abs(dw) + np.abs(self.dw0))
            if self.db is not None:
                db = db + self.db0[0]
                off_b = off_b + U32 * (np.abs(db) + np.abs(self.db0[0]))
        return (dx, dw, db), (rounded_bound(dx, off_x, self.dtype), rounded_bound(dw, off_w, self.dw_dtype),
                              rounded_bound(db, off_b, self.dw_dtype))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, dtype):
    require_gpu()
    for i, (pad, offset) in enumerate([(0, 0), (8, 0), (2, 2), (3, 1), (5, 0)]):
        act = ACTS[(i + M + K) % 5]
        acc, dw = i % 2 == 1, "f32" if i >= 3 else dtype
        what = f"linear_backward_q8 {M}x{N}x{K} {dtype} {act} pad {pad} offset {offset} dw {dw} accumulate {acc}"
        log(what)
        b = BackwardQ8(M, N, K, dtype, act, dw, acc, db=i != 1, pad=pad, offset=offset, seed=10 * i, x8=i != 2, z8=i != 0)
        b.run()
        b.check(what)


@pytest.mark.parametrize("act", ACTS)
def test_activations(act):
    require_gpu()
    for dtype in ("bf16", "f16"):
        for dw in (dtype, "f32"):
            for x8, z8 in ((True, True), (True, False), (False, True)):
                what = f"linear_backward_q8 {dtype} {act} dw {dw} x8 {x8} z8 {z8}"
                log(what)
                b = BackwardQ8(150, 264, 200, dtype, act, dw, x8=x8, z8=z8)
                b.run()
                b.check(what)


@pytest.mark.parametrize("M,N,K", LARGE)
def test_larger_sizes(M, N, K):
    require_gpu()
    for dtype, pad, dw in (("f16", 0, None), ("bf16", 6, "f32"), ("bf16", 1, None)):
        what = f"linear_backward_q8 {M}x{N}x{K} {dtype} pad {pad} dw {dw}"
        log(what)
        b = BackwardQ8(M, N, K, dtype, "gelu", dw, pad=pad)
        b.run()
        b.check(what)


def test_more_tiles_than_cus():
    require_gpu()
    M, N, K = HUGE[2]
    b = BackwardQ8(M, N, K, "bf16", "none", accumulate=True)
    log(f"linear_backward_q8 {M}x{N}x{K}")
    b.run()
    b.check(f"linear_backward_q8 {M}x{N}x{K}")


def test_each_gradient_alone():
    require_gpu()
    for keep in ("dx", "dw", "db"):
        b = BackwardQ8(90, 130, 70, "bf16", "silu")
        over = {k: None for k in ("dx", "dw", "db") if k != keep}
        if keep != "dw":
            over["x"] = None
        if keep != "dx":
            over["w"] = None
        log(f"linear_backward_q8 {keep} alone")
        b.run(**over)
        torch.cuda.synchronize()
        wants, bounds = b.bounds()
        i = ("dx", "dw", "db").index(keep)
        m = (b.dx, b.dw, b.db)[i]
        assert_close(m.f64() if keep != "db" else m.f64()[0], wants[i], bounds[i], keep)
        for other in (b.dx, b.dw, b.db):
            assert other is m or torch.isnan(other.buffer).all()


def test_without_rows():
    require_gpu()
    for accumulate in (False, True):
        log(f"linear_backward_q8 of no rows, accumulate {accumulate}")
        b = BackwardQ8(0, 40, 24, "bf16", "gelu", "f32", accumulate)
        b.run()
        b.check("no rows")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_scales_at_the_types_ends(dtype):
    """Rows of the largest and smallest scales: the codes' power of two stays in the type, the gradient's factor takes the rest."""
    require_gpu()
    log(f"linear_backward_q8 extreme scales {dtype}")
    exps = [-24, -20, -10, -1, 0, 5, 7] if dtype == "f16" else [-125, -60, -1, 0, 40, 60]
    for e in exps:
        b = BackwardQ8(40, 24, 16, dtype, "none", "f32")
        b.x.scale.view.fill_(1.5 * 2.0 ** e)
        b.x.scale.snapshot()
        b.dy.view.mul_(2.0 ** min(20, max(-40, -e)) if dtype == "bf16" else 1.0)
        b.run()
        b.check(f"scale {1.5 * 2.0 ** e}")


def test_large_gradients_in_fp16_stay_finite():
    """dy up to fp16's largest number: the factor of a row's scale is below 1."""
    require_gpu()
    log("linear_backward_q8 of large gradients")
    b = BackwardQ8(40, 24, 16, "f16", "none", "f32")
    b.dy.view.fill_(65504.0)
    b.run(dx=None, w=None)          # dx would leave fp16
    torch.cuda.synchronize()
    wants, bounds = b.bounds()
    assert_close(b.dw.f64(), wants[1], bounds[1], "dw")
    assert_close(b.db.f64()[0], wants[2], bounds[2], "db")


def test_rows_of_nan_and_of_zeros():
    """A kept row with a NaN poisons dw (every element sums over it) and nothing else; one of zeros adds nothing."""
    require_gpu()
    log("linear_backward_q8 with NaN and zero rows")
    b = BackwardQ8(90, 70, 40, "bf16", "none")
    b.x.codes.view[4] = 0
    b.x.scale.view[0, 4] = 0.0
    b.run()
    b.check("a row of zeros")
    b.x.scale.view[0, 4] = float("nan")
    b.run()
    torch.cuda.synchronize()
    assert np.isnan(b.dw.f64()).all() and np.isfinite(b.dx.f64()).all() and np.isfinite(b.db.f64()).all()


def test_without_codes_it_is_linear_backward():
    require_gpu()
    log("linear_backward_q8 without codes")
    b = Backward(150, 264, 200, "bf16", "gelu")
    b.run()
    torch.cuda.synchronize()
    first = [m.buffer.view(torch.int16).clone() for m in (b.dx, b.dw, b.db)]
    a = b.args()
    ag.linear_backward_q8(**a, workspace=workspace(ag.plan_linear_backward_q8(**a)))
    torch.cuda.synchronize()
    assert all(torch.equal(u, m.buffer.view(torch.int16)) for u, m in zip(first, (b.dx, b.dw, b.db)))


@pytest.mark.parametrize("dw", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(33, 600, 4100, 0), (513, 264, 520, 3), (1100, 8300, 600, 0), (150, 264, 200, 0), (1000, 1030, 2050, 8)])
def test_stays_inside_its_workspace(M, N, K, pad, dw):
    """On another stream than the current one, between guards, twice with the same bits."""
    require_gpu()
    side, guard = torch.cuda.Stream(), 1 << 16
    b = BackwardQ8(M, N, K, "bf16", "silu", dw, pad=pad, seed=9)
    need = ag.plan_linear_backward_q8(**b.args()).workspace_bytes
    ws = torch.full((need + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(2):
        ws[guard:guard + need] = 0xFF
        side.wait_stream(torch.cuda.current_stream())
        log(f"linear_backward_q8 {M}x{N}x{K} pad {pad} dw {dw} on a side stream")
        ag.linear_backward_q8(**b.args(), workspace=ws[guard:guard + need], stream=side)
        torch.cuda.synchronize()
        b.check(f"linear_backward_q8 {M}x{N}x{K}")
        assert bool((ws[:guard] == 0x5A).all()) and bool((ws[guard + need:] == 0x5A).all())
        bits = [m.buffer.view(torch.int32 if m.dtype == "f32" else torch.int16).clone() for m in (b.dx, b.dw, b.db)]
        assert first is None or all(torch.equal(u, v) for u, v in zip(first, bits))
        first = bits


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 520), (3, 1030, 70), (127, 4, 264), (128, 4, 264), (700, 9, 33), (2100, 64, 600), (2111, 130, 1030)])
def test_terms_of_a_wide_weight_gradient(M, N, K, dtype):
    """dw in fp32: dz's terms below each other in one product, whose stages the rows of one term end inside, or a product each."""
    require_gpu()
    for acc, pad in ((False, 0), (True, 3)):
        what = f"linear_backward_q8 {M}x{N}x{K} {dtype} dw f32 accumulate {acc} pad {pad}"
        log(what)
        b = BackwardQ8(M, N, K, dtype, "gelu_tanh", "f32", acc, pad=pad, seed=M)
        b.run()
        b.check(what)
