"""Rows in 8 bits, the root-mean-square norm and its gradients on the GPU against the float64 oracle.

Codes have to match exactly.  Bounds of the rest are per element and derived: with u = 2^-24, the norm's root is off by
half of the mean's u, u of the square root and u of the division; a product adds u, a scale's rounding u; a sum in fp32
is off by u for each addition on an element's way times the sum of magnitudes; a rounding to 16 bits is off by half a step.
Outputs lie in buffers of NaN (codes: of one byte) at odd strides and offsets, and what surrounds them has to stay.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.rows_oracle import norm_backward_oracle, norm_oracle, quantize_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import TINY, TORCH, U32, Matrix, assert_close, rounded_bound
from tests.rows_util import CodeMatrix, activations, assert_codes, vector

pytestmark = pytest.mark.gpu

EPS = 1e-6
# every kernel by its row length, whole and ragged: 16 threads a row to 1024, and rows that are read twice
SIZES = [(1, 1), (3, 7), (17, 32), (33, 100), (16, 128), (5, 129), (9, 500), (4, 512), (7, 520), (6, 1000), (5, 1024),
         (3, 1030), (2, 2048), (3, 4100), (1, 4096), (3, 8191), (1, 8192), (2, 10000), (2, 16384), (2, 20001), (1, 32768),
         (2, 33000), (1, 70001)]
LAYOUTS = [(0, 0), (8, 0), (3, 1)]          # pads and offsets of rows


def f64(t):
    return t.double().cpu().numpy()


def rounded_sum(x, r, dtype):
    """x + r rounded once to dtype (float32 holds enough bits on the way for that)."""
    return (x.double() + r.double()).to(TORCH[dtype])


class Norm:
    def __init__(self, M, K, dtype, x=None, weight=True, residual=True, h=True, y=True, q=True, rstd=True, pad=0, offset=0, seed=1):
        self.shape, self.dtype = (M, K), dtype
        mat = lambda values=None: Matrix(M, K, dtype, pad=pad, offset=offset, values=values)  # noqa: E731
        self.x0 = activations(seed, M, K, dtype) if x is None else x
        self.r0 = activations(seed + 1, M, K, dtype) if residual else None
        g = np.random.default_rng(seed)
        self.w0 = torch.from_numpy(1 + 0.2 * g.standard_normal(K)).to(TORCH[dtype]) if weight else None
        self.x = mat(self.x0)
        self.r = mat(self.r0) if residual else None
        self.w = Matrix(1, K, dtype, offset=offset, values=self.w0[None, :]) if weight else None
        self.h, self.y = mat() if h else None, mat() if y else None
        self.q = CodeMatrix(M, K, pad=pad, offset=offset) if q else None
        self.scale = vector(M, offset) if q else None
        self.rstd = vector(M, offset) if rstd else None

    def args(self):
        M, K = self.shape
        at = lambda m: m.ptr if m is not None else None  # noqa: E731
        ld = lambda m: m.ld if m is not None else 0  # noqa: E731
        return dict(x=self.x.ptr, M=M, K=K, dtype=self.dtype, weight=at(self.w), residual=at(self.r), h=at(self.h), y=at(self.y),
                    q=at(self.q), scale=at(self.scale), rstd=at(self.rstd), eps=EPS, ldx=self.x.ld, ldr=ld(self.r), ldh=ld(self.h),
                    ldy=ld(self.y), ldq=ld(self.q))

    def check(self, what):
        torch.cuda.synchronize()
        h0 = self.x0 if self.r0 is None else rounded_sum(self.x0, self.r0, self.dtype)
        y, rstd, codes, scale = norm_oracle(f64(h0), f64(self.w0) if self.w0 is not None else None, EPS)
        if self.h is not None:
            assert torch.equal(self.h.view.cpu(), h0), f"{what} h"
        if self.rstd is not None:
            assert_close(self.rstd.f64()[0], rstd, 2.5 * U32 * rstd, f"{what} rstd")
        if self.y is not None:
            assert_close(self.y.f64(), y, rounded_bound(y, 3.6 * U32 * np.abs(y), self.dtype), f"{what} y")
        if self.q is not None:
            assert_codes(self.q.numpy(), codes, f"{what} codes")
            assert_close(self.scale.f64()[0], scale, 3.6 * U32 * scale + TINY["f32"], f"{what} scale")
        for name in ("x", "r", "w", "h", "y", "q", "scale", "rstd"):
            m = getattr(self, name)
            if m is not None:
                m.check_surroundings(f"{what} {name}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_sizes(M, K, dtype):
    require_gpu()
    for pad, offset in LAYOUTS:
        what = f"norm {M}x{K} {dtype} pad {pad} offset {offset}"
        log(what)
        n = Norm(M, K, dtype, pad=pad, offset=offset)
        ag.rms_norm(**n.args())
        n.check(what)


@pytest.mark.parametrize("K", [96, 520, 4100, 40000])
def test_norm_parts(K):
    """Each output alone, and each input left out."""
    require_gpu()
    parts = [dict(y=False, q=False), dict(h=False, y=False), dict(h=False, q=False, rstd=False), dict(residual=False),
             dict(weight=False), dict(residual=False, h=False, weight=False, q=False), dict(y=False, q=False, rstd=False)]
    for i, part in enumerate(parts):
        what = f"norm 5x{K} {part}"
        log(what)
        n = Norm(5, K, "bf16" if i % 2 else "f16", pad=3, **part)
        ag.rms_norm(**n.args())
        n.check(what)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("K", [64, 520, 4096, 9000, 40000])
def test_norm_in_place(K, which):
    """h may be x or the residual."""
    require_gpu()
    log(f"norm 6x{K}: h is {which}")
    n = Norm(6, K, "bf16", pad=2)
    inside = n.x if which == "x" else n.r
    n.h = inside
    ag.rms_norm(**n.args())
    n.check(f"norm 6x{K} in place of {which}")


def test_norm_many_rows():
    """More rows than a launch's workgroups hold at a time."""
    require_gpu()
    for M, K, dtype in ((70001, 64, "bf16"), (9001, 300, "f16"), (9001, 1000, "bf16"), (2500, 2050, "f16"), (700, 16384, "bf16")):
        log(f"norm {M}x{K} {dtype}")
        n = Norm(M, K, dtype)
        ag.rms_norm(**n.args())
        n.check(f"norm {M}x{K}")


def special_rows(dtype, K):
    """Rows of zeros, of the type's extremes, with NaN and infinities, of one element, and full of ties."""
    x = torch.zeros(12, K, dtype=torch.float64)
    big, small = torch.finfo(TORCH[dtype]).max, torch.finfo(TORCH[dtype]).smallest_normal
    g = np.random.default_rng(5)
    x[1] = torch.from_numpy(g.standard_normal(K))
    x[1, K // 2] = float("nan")
    x[2] = 1.0
    x[2, K - 1] = float("inf")
    x[3, 0] = float("-inf")
    x[4, K - 1] = -3.0
    x[5] = torch.from_numpy(g.integers(-127, 128, K).astype(np.float64))      # 254 halves: every odd number is a tie
    x[5, 0] = 254.0
    x[6] = torch.from_numpy(g.standard_normal(K)) * 2.0 ** (60 if dtype == "bf16" else 12)
    x[7] = torch.from_numpy(g.standard_normal(K)) * 2.0 ** (-60 if dtype == "bf16" else -12)
    x[8] = big / 2
    x[9] = small
    x[10] = torch.from_numpy(g.integers(-127, 128, K).astype(np.float64)) * 0.5 + 0.25
    x[10, 0] = -127.0
    x[11] = 127.0
    return x.to(TORCH[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("K", [24, 130, 600, 1500, 5000, 9000, 35000])
def test_norm_special_rows(K, dtype):
    """Without a weight, so that ties stay ties."""
    require_gpu()
    log(f"norm special rows, K {K} {dtype}")
    x = special_rows(dtype, K)
    n = Norm(12, K, dtype, x=x, weight=False, residual=False, h=False)
    ag.rms_norm(**n.args())
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        y, rstd, codes, scale = norm_oracle(f64(x), None, EPS)
    assert_codes(n.q.numpy(), codes, "codes")
    got_y, got_rstd, got_scale = n.y.f64(), n.rstd.f64()[0], n.scale.f64()[0]
    fine = [0, 4, 5, 6, 7, 8, 9, 10, 11]
    assert_close(got_rstd[fine], rstd[fine], 2.5 * U32 * rstd[fine], "rstd")
    assert_close(got_scale[fine], scale[fine], 3.6 * U32 * scale[fine] + TINY["f32"], "scale")
    assert_close(got_y[fine], y[fine], rounded_bound(y[fine], 3.6 * U32 * np.abs(y[fine]), dtype), "y")
    assert np.isnan(got_scale[[1, 2, 3]]).all() and np.isnan(got_y[1]).all() and np.isnan(got_y[2, K - 1]) and np.isnan(got_y[3, 0])


@pytest.mark.parametrize("K", [40, 1000, 5000, 40000])
def test_norm_products_past_fp32(K):
    """h weight past fp32's largest: an infinity in y, the row's scale NaN and its codes 0; the sums keep their range."""
    require_gpu()
    log(f"norm of products past fp32, K {K}")
    x = torch.ones(3, K, dtype=torch.bfloat16)
    x[1] = 2.0 ** 120
    n = Norm(3, K, "bf16", x=x, residual=False)
    n.w.view.fill_(1.0)
    n.w.view[0, K - 1] = 2.0 ** 20
    n.w.snapshot()
    ag.rms_norm(**n.args())
    torch.cuda.synchronize()
    y, q, s, r = n.y.f64(), n.q.numpy(), n.scale.f64()[0], n.rstd.f64()[0]
    assert np.isposinf(y[1, K - 1]) and np.isfinite(y[1, :-1]).all() and np.isnan(s[1]) and not q[1].any()
    assert np.isfinite(y[[0, 2]]).all() and np.isfinite(s[[0, 2]]).all() and (q[[0, 2], K - 1] == 127).all()
    assert abs(r[1] * 2.0 ** 120 - 1) <= 2.5 * U32


# ------------------------------------------------------------------ codes

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,K", SIZES)
def test_quantize_and_back(M, K, dtype):
    require_gpu()
    for pad, offset in LAYOUTS:
        what = f"codes {M}x{K} {dtype} pad {pad} offset {offset}"
        log(what)
        x = activations(3, M, K, dtype)
        m, q, s = Matrix(M, K, dtype, pad=pad, offset=offset, values=x), CodeMatrix(M, K, pad=pad, offset=offset), vector(M, offset)
        y = Matrix(M, K, dtype, pad=pad, offset=offset)
        ag.quantize_rows(m.ptr, q.ptr, s.ptr, M, K, dtype, ldx=m.ld, ldq=q.ld)
        ag.dequantize_rows(q.ptr, s.ptr, y.ptr, M, K, dtype, ldq=q.ld, ldy=y.ld)
        torch.cuda.synchronize()
        codes, scale = quantize_oracle(f64(x))
        assert_codes(q.numpy(), codes, what)
        got = s.f64()[0]
        assert_close(got, scale, U32 * (1 + 2.0 ** -20) * scale + TINY["f32"], f"{what} scale")
        back = codes * got[:, None]
        # an fp32 product, and for 16 bits its rounding
        bound = U32 * np.abs(back) + TINY["f32"] if dtype == "f32" else rounded_bound(back, U32 * np.abs(back), dtype)
        assert_close(y.f64(), back, bound, f"{what} values")
        for t in (m, q, s, y):
            t.check_surroundings(what)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("K", [24, 130, 600, 1500, 5000, 9000, 35000])
def test_quantize_special_rows(K, dtype):
    require_gpu()
    log(f"codes of special rows, K {K} {dtype}")
    x = special_rows(dtype, K)
    if dtype == "f32":          # the ends of fp32, subnormal numbers among them
        x[9] = 2.0 ** -149
        x[6] *= 2.0 ** 80
        x[7] *= 2.0 ** -130
    q, s = CodeMatrix(12, K), vector(12)
    m = Matrix(12, K, dtype, values=x)
    ag.quantize_rows(m.ptr, q.ptr, s.ptr, 12, K, dtype)
    torch.cuda.synchronize()
    codes, scale = quantize_oracle(f64(x))
    assert_codes(q.numpy(), codes, f"K {K} {dtype}")
    got = s.f64()[0]
    bad = np.isnan(scale)
    assert bad.tolist() == [i in (1, 2, 3) for i in range(12)] and np.isnan(got[bad]).all()
    assert_close(got[~bad], scale[~bad], U32 * (1 + 2.0 ** -20) * scale[~bad] + 2 * TINY["f32"], "scale")


def test_rows_without_elements():
    require_gpu()
    log("rows of no elements, no rows")
    s, r = vector(5), vector(5)
    ag.quantize_rows(None, None, s.ptr, 5, 0, "bf16")
    ag.rms_norm(None, 5, 0, "bf16", rstd=r.ptr, eps=4.0)
    ag.quantize_rows(None, None, None, 0, 64, "bf16")
    ag.rms_norm(None, 0, 64, "f16")
    ag.dequantize_rows(None, s.ptr, None, 5, 0, "f16")
    torch.cuda.synchronize()
    assert s.f64()[0].tolist() == [0.0] * 5 and r.f64()[0].tolist() == [0.5] * 5


def test_rows_far_apart():
    """Offsets past 2^32 bytes: the last rows of a matrix whose rows lie 2^20 elements apart."""
    require_gpu()
    M, K, ld = 2200, 40, 1 << 20
    log(f"norm {M}x{K} at stride {ld}")
    x = torch.zeros((M - 1) * ld + K, dtype=torch.bfloat16, device="cuda").as_strided((M, K), (ld, 1))
    x0 = activations(9, M, K, "bf16")
    x.copy_(x0)
    y = torch.zeros((M - 1) * ld + K, dtype=torch.bfloat16, device="cuda").as_strided((M, K), (ld, 1))
    q = torch.zeros((M - 1) * ld + K, dtype=torch.int8, device="cuda").as_strided((M, K), (ld, 1))
    s = torch.empty(M, device="cuda")
    ag.rms_norm(x, M, K, "bf16", y=y, q=q, scale=s, eps=EPS, ldx=ld, ldy=ld, ldq=ld)
    torch.cuda.synchronize()
    want, _, codes, scale = norm_oracle(f64(x0), None, EPS)
    assert_codes(q.cpu().numpy(), codes, "codes")
    assert_close(f64(y), want, rounded_bound(want, 3.6 * U32 * np.abs(want), "bf16"), "y")
    assert_close(f64(s), scale, 3.6 * U32 * scale, "scale")
    ag.dequantize_rows(q, s, y, M, K, "bf16", ldq=ld, ldy=ld)
    torch.cuda.synchronize()
    back = codes * f64(s)[:, None]
    assert_close(f64(y), back, rounded_bound(back, U32 * np.abs(back), "bf16"), "values")


# ------------------------------------------------------------------ gradients of the norm

class Backward:
    def __init__(self, M, K, dtype, dw="f32", weight=True, dh=True, accumulate=False, pad=0, offset=0, seed=1, dx=True, want_dw=True):
        self.shape, self.dtype, self.dwt, self.accumulate = (M, K), dtype, dw, accumulate
        mat = lambda values=None: Matrix(M, K, dtype, pad=pad, offset=offset, values=values)  # noqa: E731
        g = np.random.default_rng(seed)
        normal = lambda *s: torch.from_numpy(g.standard_normal(s)).to(TORCH[dtype])  # noqa: E731
        self.h0, self.dy0 = activations(seed, M, K, dtype), normal(M, K)
        self.dh0 = normal(M, K) if dh else None
        self.w0 = torch.from_numpy(1 + 0.2 * g.standard_normal(K)).to(TORCH[dtype]) if weight else None
        self.rstd0 = 1 / np.sqrt((f64(self.h0) ** 2).mean(1) + EPS)
        self.rstd0 = self.rstd0.astype(np.float32)
        self.before = g.standard_normal(K).astype(np.float32)
        self.h, self.dy = mat(self.h0), mat(self.dy0)
        self.dh = mat(self.dh0) if dh else None
        self.w = Matrix(1, K, dtype, offset=offset, values=self.w0[None, :]) if weight else None
        self.rstd = vector(M, offset, self.rstd0)
        self.dx = mat() if dx else None
        self.dw = Matrix(1, K, dw, offset=offset, values=torch.from_numpy(self.before)[None, :] if accumulate else None) if want_dw else None
        if accumulate:
            self.before = self.dw.f64()[0]

    def args(self):
        M, K = self.shape
        at = lambda m: m.ptr if m is not None else None  # noqa: E731
        ld = lambda m: m.ld if m is not None else 0  # noqa: E731
        return dict(dy=self.dy.ptr, h=self.h.ptr, rstd=self.rstd.ptr, M=M, K=K, dtype=self.dtype, weight=at(self.w), dh=at(self.dh),
                    dx=at(self.dx), dw=at(self.dw), lddy=self.dy.ld, ldh=self.h.ld, lddh=ld(self.dh), lddx=ld(self.dx),
                    dw_dtype=self.dwt, accumulate=self.accumulate)

    def run(self, stream=None):
        p = ag.plan_rms_norm_backward(**self.args())
        ws = torch.full((p.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda") if p.workspace_bytes else None
        ag.rms_norm_backward(**self.args(), workspace=ws, stream=stream)
        return p

    def check(self, what, plan):
        torch.cuda.synchronize()
        M, K = self.shape
        h, dy, r = f64(self.h0), f64(self.dy0), self.rstd0.astype(np.float64)
        w = f64(self.w0) if self.w0 is not None else np.ones(K)
        dh = f64(self.dh0) if self.dh0 is not None else None
        dx, dw = norm_backward_oracle(dy, h, r, w, dh)
        n, g = h * r[:, None], dy * w
        if self.dx is not None:
            # additions on an element's way: of a thread one after the other, 6 in a wave, up to 16 waves
            adds = 8 * max(1, plan.vectors_per_thread or -(-K // 8192)) + 22
            c = np.abs((g * n).sum(1) / K)[:, None]
            c_off = (adds + 4) * U32 * np.abs(g * n).sum(1)[:, None] / K
            off = r[:, None] * ((np.abs(g) + np.abs(n) * c) * 4 * U32 + np.abs(n) * c_off) + (U32 * np.abs(dx))
            assert_close(self.dx.f64(), dx, rounded_bound(dx, off, self.dtype), f"{what} dx")
            self.dx.check_surroundings(f"{what} dx")
        if self.dw is not None:
            if plan.launches == 1:      # little work: 32 lanes down the rows, then over the lanes
                adds = -(-M // 32) + 32
            else:                       # a thread's rows, a workgroup's threads, the workgroups in 32 lanes, the lanes
                rows = max(1, 256 // plan.threads_per_row) if plan.threads_per_row else 1
                adds = -(-M // max(1, plan.n_programs * rows)) + rows + -(-plan.n_programs // 32) + 32
            off = (adds + 3) * U32 * np.abs(dy * n).sum(0)
            if self.accumulate:
                dw = dw + self.before
                off = off + U32 * np.abs(dw)
            bound = off + TINY["f32"] if self.dwt == "f32" else rounded_bound(dw, off, self.dwt)
            assert_close(self.dw.f64()[0], dw, bound, f"{what} dw")
            self.dw.check_surroundings(f"{what} dw")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_backward_sizes(M, K, dtype):
    require_gpu()
    for i, (pad, offset) in enumerate(LAYOUTS):
        what = f"norm backward {M}x{K} {dtype} pad {pad} offset {offset}"
        log(what)
        b = Backward(M, K, dtype, "f32" if i % 2 else dtype, pad=pad, offset=offset, accumulate=i == 2, dh=i != 1, weight=i != 1)
        b.check(what, b.run())


@pytest.mark.parametrize("M,K,dtype", [(511, 1000, "bf16"), (512, 4096, "f16"), (513, 4096, "bf16"), (70001, 64, "bf16"), (9001, 300, "f16"), (9001, 1000, "bf16"), (5000, 2050, "f16"),
                                       (1200, 16384, "bf16"), (520, 40000, "f16")])
def test_norm_backward_many_rows(M, K, dtype):
    require_gpu()
    log(f"norm backward {M}x{K} {dtype}")
    b = Backward(M, K, dtype, "f32")
    b.check(f"norm backward {M}x{K}", b.run())


@pytest.mark.parametrize("K", [64, 520, 4100, 40000])
def test_norm_backward_parts(K):
    """dx or dw alone; dx in place of dh."""
    require_gpu()
    for part in (dict(dx=False), dict(want_dw=False), dict(dx=False, dh=False, weight=False)):
        what = f"norm backward 21x{K} {part}"
        log(what)
        b = Backward(21, K, "bf16", **part)
        b.check(what, b.run())
    b = Backward(21, K, "f16")
    b.dx = b.dh
    log(f"norm backward 21x{K} in place")
    b.check(f"norm backward 21x{K} in place", b.run())


def test_norm_backward_without_rows():
    require_gpu()
    log("norm backward of no rows")
    for dw, accumulate in (("bf16", False), ("f32", False), ("f32", True)):
        b = Backward(0, 100, "bf16", dw, accumulate=accumulate)
        b.run()
        torch.cuda.synchronize()
        assert np.array_equal(b.dw.f64()[0], b.before if accumulate else np.zeros(100))


def test_norm_gradients_against_differences():
    """The definition's gradients against differences of the definition, and the kernel's against both."""
    require_gpu()
    log("norm gradients against differences")
    M, K = 3, 40
    b = Backward(M, K, "f16", "f32", dh=False)
    p = b.run()
    b.check("norm backward", p)
    h, w, dy = f64(b.h0), f64(b.w0), f64(b.dy0)
    loss = lambda hh, ww: (norm_oracle(hh, ww, EPS)[0] * dy).sum()  # noqa: E731
    step = 1e-5
    rstd = 1 / np.sqrt((h ** 2).mean(1) + EPS)
    dx, dw = norm_backward_oracle(dy, h, rstd, w)
    for i in range(M):
        for k in range(0, K, 7):
            d = np.zeros_like(h)
            d[i, k] = step
            assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * step) - dx[i, k]) < 1e-7
    for k in range(0, K, 5):
        d = np.zeros(K)
        d[k] = step
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * step) - dw[k]) < 1e-7


# ------------------------------------------------------------------ streams, graphs, workspaces

def test_norm_backward_stays_inside_its_workspace():
    """On another stream than the current one, twice with the same bits."""
    require_gpu()
    side = torch.cuda.Stream()
    for M, K in ((80, 520), (3000, 4100), (5000, 100)):
        b = Backward(M, K, "bf16", "f32", pad=3)
        plan = ag.plan_rms_norm_backward(**b.args())
        ws = torch.full((plan.workspace_bytes + (2 << 16),), 0x5A, dtype=torch.uint8, device="cuda")
        first = None
        for _ in range(2):
            side.wait_stream(torch.cuda.current_stream())
            log(f"norm backward {M}x{K} on a side stream")
            ag.rms_norm_backward(**b.args(), workspace=ws[1 << 16:-(1 << 16)], stream=side)
            torch.cuda.synchronize()
            b.check(f"norm backward {M}x{K}", plan)
            assert bool((ws[:1 << 16] == 0x5A).all()) and bool((ws[-(1 << 16):] == 0x5A).all())
            bits = [b.dx.buffer.view(torch.int16).clone(), b.dw.buffer.view(torch.int32).clone()]
            assert first is None or all(torch.equal(u, v) for u, v in zip(first, bits))
            first = bits


def test_rows_in_a_graph():
    """Captured once and replayed on new inputs, with eager work and synchronizations in between."""
    require_gpu()
    log("rows in a graph")
    M, K = 300, 1000
    x, y = (torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dx, h, back = (torch.empty_like(x) for _ in range(3))
    q, s, r = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    w, dw = torch.ones(K, dtype=torch.bfloat16, device="cuda"), torch.empty(K, device="cuda")
    nbytes = ag.plan_rms_norm_backward(y, h, r, M, K, "bf16", w, x, dx, dw, dw_dtype="f32").workspace_bytes
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def step(stream):
        ag.rms_norm(x, M, K, "bf16", w, x, h, y, q, s, r, stream=stream)
        ag.dequantize_rows(q, s, back, M, K, "bf16", stream=stream)
        ag.rms_norm_backward(y, h, r, M, K, "bf16", w, x, dx, dw, dw_dtype="f32", workspace=ws, stream=stream)

    outputs = (h, y, q, s, r, back, dx, dw)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    x.copy_(activations(1, M, K, "bf16"))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for i in range(4):
        x.copy_(activations(10 + i, M, K, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outputs]
        step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, outputs)), f"replay {i}"


def test_two_streams_at_once():
    """Calls that may run side by side, each with a workspace of its own."""
    require_gpu()
    log("norm gradients on two streams")
    work = []
    for i, (M, K) in enumerate(((3000, 4100), (4000, 1000), (300, 600), (900, 20000))):
        b = Backward(M, K, "bf16", "f32", seed=20 + i)
        p = ag.plan_rms_norm_backward(**b.args())
        work.append((b, p, torch.full((max(1, p.workspace_bytes),), 0xA5, dtype=torch.uint8, device="cuda")))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (b, p, ws) in enumerate(work):
            ag.rms_norm_backward(**b.args(), workspace=ws, stream=streams[i % 2])
    torch.cuda.synchronize()
    for b, p, _ in work:
        b.check(f"norm backward {b.shape} beside others", p)
