"""The linear layer and its gradients on the GPU against the float64 oracle.

Bounds are per element and derived: an fp32 sum of K products is off by at
most (K + 8) 2^-24 times the sum of their magnitudes, an activation's fp32
evaluation by 2^-19 of its argument's size, and a rounding by half a step.
Inputs and outputs lie in buffers of NaN, so that reading a pad poisons the
result and writing one is seen.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import act_oracle, linear_backward_oracle, linear_oracle, slope_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import (ACT_ERROR, HALF_STEP, HUGE, LARGE, U32, Matrix, TORCH, assert_close, product_bound, random_matrix,
                               rounded_bound)

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def workspace(plan):
    return torch.full((plan.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda") if plan.workspace_bytes else None


class Forward:
    def __init__(self, M, N, K, dtype, act="none", bias=True, residual=True, z=True, pad=0, offset=0, seed=1):
        self.shape, self.dtype, self.act = (M, N, K), dtype, act
        self.x = random_matrix(seed, M, K, dtype, pad=pad, offset=offset)
        self.w = random_matrix(seed + 1, N, K, dtype, 1 / np.sqrt(max(K, 1)), pad=pad, offset=offset)
        self.b = random_matrix(seed + 2, 1, N, dtype, 0.5, offset=offset) if bias else None
        self.r = random_matrix(seed + 3, M, N, dtype, pad=pad, offset=offset) if residual else None
        self.y = Matrix(M, N, dtype, pad=pad, offset=offset)
        self.z = Matrix(M, N, dtype, pad=pad, offset=offset) if z else None

    def args(self):
        M, N, K = self.shape
        at = lambda m: m.ptr if m is not None else None  # noqa: E731
        ld = lambda m: m.ld if m is not None else 0  # noqa: E731
        return dict(x=self.x.ptr, w=self.w.ptr, y=self.y.ptr, M=M, N=N, K=K, dtype=self.dtype, act=self.act,
                    bias=at(self.b), residual=at(self.r), z=at(self.z), ldx=self.x.ld, ldw=self.w.ld, ldr=ld(self.r),
                    ldy=self.y.ld, ldz=ld(self.z))

    def run(self, stream=None, **over):
        a = dict(self.args(), **over)
        ag.linear(**a, workspace=workspace(ag.plan_linear(**a)), stream=stream)

    def check(self, what, residual=None):
        torch.cuda.synchronize()
        M, N, K = self.shape
        x, w = self.x.f64(), self.w.f64()
        b = self.b.f64()[0] if self.b is not None else None
        r = residual if residual is not None else self.r.f64() if self.r is not None else None
        y, z = linear_oracle(x, w, b, self.act, r)
        off = product_bound(x, w, K) + U32 * (np.abs(z) + (np.abs(b) if b is not None else 0))
        if self.z is not None:
            assert_close(self.z.f64(), z, rounded_bound(z, off, self.dtype), what + " z")
            self.z.check_surroundings(what + " z")
        # no slope is above 1.13
        off = 1.13 * off + ACT_ERROR * np.abs(z) + U32 * (np.abs(y) + (np.abs(r) if r is not None else 0))
        assert_close(self.y.f64(), y, rounded_bound(y, off, self.dtype), what + " y")
        self.y.check_surroundings(what + " y")


SIZES = [(1, 1, 1), (1, 16, 128), (1, 15, 7), (2, 17, 129), (3, 520, 136), (13, 130, 1000), (16, 64, 64), (17, 33, 65),
         (32, 100, 260), (33, 16, 63), (33, 1, 64), (40, 130, 1), (64, 8, 66), (80, 136, 128), (129, 127, 200),
         (128, 128, 192), (200, 257, 100), (257, 300, 520)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_sizes(M, N, K, dtype):
    require_gpu()
    for i, (pad, offset) in enumerate([(0, 0), (8, 0), (2, 2), (3, 1), (5, 0)]):
        act = ACTS[(i + M + N) % 5]
        what = f"linear {M}x{N}x{K} {dtype} {act} pad {pad} offset {offset}"
        log(what)
        f = Forward(M, N, K, dtype, act, pad=pad, offset=offset, seed=10 * i)
        f.run()
        f.check(what)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 70])
def test_linear_epilogue_parts(M, act):
    require_gpu()
    for bias in (False, True):
        for residual in (False, True):
            for z in (False, True):
                what = f"linear {M} {act} bias {bias} residual {residual} z {z}"
                log(what)
                f = Forward(M, 200, 96, "bf16", act, bias, residual, z, pad=4)
                f.run()
                f.check(what)




@pytest.mark.parametrize("M,N,K", LARGE)
def test_linear_larger_sizes(M, N, K):
    require_gpu()
    for dtype, pad in (("f16", 0), ("bf16", 6), ("bf16", 1)):
        what = f"linear {M}x{N}x{K} {dtype} pad {pad}"
        log(what)
        f = Forward(M, N, K, dtype, "gelu_tanh", pad=pad)
        p = ag.plan_linear(**f.args())
        log(f"  tile {p.product.tile_m}x{p.product.tile_n} full {p.product.full_tiles} of {p.product.n_programs} programs packed {p.product.packed}")
        f.run()
        f.check(what)


def test_linear_more_tiles_than_cus():
    """Whole rounds of tiles, and the others' reductions cut."""
    require_gpu()
    M, N, K = HUGE[0]
    f = Forward(M, N, K, "bf16", "silu", z=False)
    p = ag.plan_linear(**f.args()).product
    log(f"linear {M}x{N}x{K}: tile {p.tile_m}x{p.tile_n} full {p.full_tiles} splits {p.splits}")
    f.run()
    f.check(f"linear {M}x{N}x{K}")


@pytest.mark.parametrize("M", [0, 1, 40])
def test_linear_without_reduction_or_output(M):
    """K = 0 leaves act(bias) + residual; M = 0 or N = 0 nothing to do."""
    require_gpu()
    for N, K in ((24, 0), (0, 24), (24, 24), (0, 0)):
        if M and N and K:
            continue
        log(f"linear {M}x{N}x{K}")
        f = Forward(M, N, K, "f16", "silu")
        f.run()
        f.check(f"linear {M}x{N}x{K}")


@pytest.mark.parametrize("M", [3, 300])
def test_linear_residual_in_place(M):
    require_gpu()
    f = Forward(M, 264, 128, "bf16", "gelu", residual=True)
    r = f.r.f64()
    f.y.view.copy_(f.r.view)
    f.y.snapshot()
    log(f"linear in place {M}")
    f.run(residual=f.y.ptr, ldr=f.y.ld)
    f.check("linear in place", residual=r)


@pytest.mark.parametrize("M", [2, 100])
def test_linear_infinities_and_nan_stay_in_their_rows(M):
    require_gpu()
    f = Forward(M, 70, 130, "f16", "none", residual=False)
    f.x.view[1, 129] = float("inf")
    f.w.view[69, 0] = float("nan")
    log(f"linear non-finite {M}")
    f.run()
    torch.cuda.synchronize()
    y, want = f.y.f64(), linear_oracle(f.x.f64(), f.w.f64(), f.b.f64()[0])[0]
    assert np.array_equal(np.isnan(y), np.isnan(want))
    assert np.array_equal(np.isinf(y), np.isinf(want))


@pytest.mark.parametrize("M", [1, 33, 513])
def test_linear_on_another_stream_twice_the_same(M):
    require_gpu()
    f = Forward(M, 520, 2048, "bf16", "silu")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    log(f"linear on a side stream, {M} rows")
    f.run(stream=side)
    f.check("linear, side stream")
    first = f.y.buffer.view(torch.int16).clone()
    f.run(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(first, f.y.buffer.view(torch.int16))


def test_linear_offsets_beyond_32_bits():
    """x of 2^31 elements and more: its last rows, through the tiles and as the reduction of dw."""
    require_gpu()
    M, N, K = 262200, 40, 8200
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = (torch.randn(N, K, generator=g, device="cuda") / K ** 0.5).bfloat16()
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert M * K > 2 ** 31
    args = dict(x=x, w=w, y=y, M=M, N=N, K=K, dtype="bf16")
    log("linear beyond 2^31 elements")
    ag.linear(**args, workspace=workspace(ag.plan_linear(**args)))
    torch.cuda.synchronize()
    for first in (0, 131000, 261900, M - 7):
        xs = x[first:first + 7].double().cpu().numpy()
        want = xs @ w.double().cpu().numpy().T
        bound = rounded_bound(want, product_bound(xs, w.double().cpu().numpy(), K), "bf16")
        assert_close(y[first:first + 7].double().cpu().numpy(), want, bound, f"rows from {first}")
    # dw of a gradient that is zero but in the last rows is their product alone
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dy[-5:] = torch.randn(5, N, generator=g, device="cuda").bfloat16()
    dw = torch.empty(N, K, dtype=torch.float32, device="cuda")
    args = dict(dy=dy, x=x, w=None, M=M, N=N, K=K, dtype="bf16", dw=dw, dw_dtype="f32")
    log("linear_backward beyond 2^31 elements")
    ag.linear_backward(**args, workspace=workspace(ag.plan_linear_backward(**args)))
    torch.cuda.synchronize()
    d, xs = dy[-5:].double().cpu().numpy(), x[-5:].double().cpu().numpy()
    assert_close(dw.double().cpu().numpy(), d.T @ xs, product_bound(d.T, xs.T, 5) + 1e-30, "dw")


# ------------------------------------------------------------------ gradients

class Backward:
    def __init__(self, M, N, K, dtype, act="none", dw_dtype=None, accumulate=False, db=True, pad=0, offset=0, seed=1):
        self.shape, self.dtype, self.act, self.accumulate = (M, N, K), dtype, act, accumulate
        self.dw_dtype = dw_dtype or dtype
        self.dy = random_matrix(seed, M, N, dtype, pad=pad, offset=offset)
        self.z = random_matrix(seed + 1, M, N, dtype, 2.0, pad=pad, offset=offset) if act != "none" else None
        self.x = random_matrix(seed + 2, M, K, dtype, pad=pad, offset=offset)
        self.w = random_matrix(seed + 3, N, K, dtype, 1 / np.sqrt(max(N, 1)), pad=pad, offset=offset)
        self.dx = Matrix(M, K, dtype, pad=pad, offset=offset)
        g = random_matrix if accumulate else (lambda s, r, c, t, **kw: Matrix(r, c, t, **kw))
        self.dw = g(seed + 4, N, K, self.dw_dtype, pad=pad, offset=offset)
        self.db = g(seed + 5, 1, N, self.dw_dtype, offset=offset) if db else None
        self.dw0, self.db0 = self.dw.f64(), self.db.f64() if db else None

    def args(self):
        M, N, K = self.shape
        return dict(dy=self.dy.ptr, x=self.x.ptr, w=self.w.ptr, M=M, N=N, K=K, dtype=self.dtype, act=self.act,
                    z=self.z.ptr if self.z else None, dx=self.dx.ptr, dw=self.dw.ptr,
                    db=self.db.ptr if self.db else None, lddy=self.dy.ld, ldx=self.x.ld, ldw=self.w.ld,
                    ldz=self.z.ld if self.z else 0, lddx=self.dx.ld, lddw=self.dw.ld, dw_dtype=self.dw_dtype,
                    accumulate=self.accumulate)

    def run(self, stream=None, **over):
        a = dict(self.args(), **over)
        ag.linear_backward(**a, workspace=workspace(ag.plan_linear_backward(**a)), stream=stream)

    def bounds(self):
        """(wants, bounds) of dx, dw, db."""
        M, N, K = self.shape
        dy, x, w = self.dy.f64(), self.x.f64(), self.w.f64()
        z = self.z.f64() if self.z else np.zeros_like(dy)
        dx, dw, db, dz = linear_backward_oracle(dy, z, x, w, self.act)
        # dz: evaluated in fp32, then one rounding for the products
        dz_off = (ACT_ERROR * (1 + np.abs(z)) + U32) * np.abs(dy) if self.act != "none" else np.zeros_like(dy)
        dz_rounded = rounded_bound(dz, dz_off, self.dtype) if self.act != "none" else dz_off
        size = np.abs(dz) + dz_rounded
        off_x = dz_rounded @ np.abs(w) + (N + 8) * U32 * (size @ np.abs(w))
        off_w = dz_rounded.T @ np.abs(x) + (M + 8) * U32 * (size.T @ np.abs(x))
        off_b = dz_off.sum(0) + (M + 8) * U32 * size.sum(0)
        if self.accumulate:
            dw = dw + self.dw0
            off_w = off_w + U32 * (np.abs(dw) + np.abs(self.dw0))
            if self.db is not None:
                db = db + self.db0[0]
                off_b = off_b + U32 * (np.abs(db) + np.abs(self.db0[0]))
        return (dx, dw, db), (rounded_bound(dx, off_x, self.dtype), rounded_bound(dw, off_w, self.dw_dtype),
                              rounded_bound(db, off_b, self.dw_dtype))

    def check(self, what):
        torch.cuda.synchronize()
        wants, bounds = self.bounds()
        got = (self.dx.f64(), self.dw.f64(), self.db.f64()[0] if self.db else wants[2])
        for name, g, want, bound in zip(("dx", "dw", "db"), got, wants, bounds):
            assert_close(g, want, bound, f"{what} {name}")
        for m in (self.dx, self.dw, self.db):
            if m is not None:
                m.check_surroundings(what)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_backward_sizes(M, N, K, dtype):
    require_gpu()
    for i, (pad, offset) in enumerate([(0, 0), (8, 0), (2, 2), (3, 1), (5, 0)]):
        act = ACTS[(i + M + K) % 5]
        acc, dw = i % 2 == 1, "f32" if i >= 3 else dtype
        what = f"linear_backward {M}x{N}x{K} {dtype} {act} pad {pad} offset {offset} dw {dw} accumulate {acc}"
        log(what)
        b = Backward(M, N, K, dtype, act, dw, acc, db=i != 1, pad=pad, offset=offset, seed=10 * i)
        b.run()
        b.check(what)


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_activations(act):
    require_gpu()
    for dw in ("bf16", "f32"):
        log(f"linear_backward {act} dw {dw}")
        b = Backward(150, 264, 200, "bf16", act, dw)
        b.run()
        b.check(f"linear_backward {act} dw {dw}")


@pytest.mark.parametrize("M,N,K", LARGE)
def test_linear_backward_larger_sizes(M, N, K):
    require_gpu()
    for dtype, pad in (("f16", 0), ("bf16", 6), ("bf16", 1)):
        what = f"linear_backward {M}x{N}x{K} {dtype} pad {pad}"
        log(what)
        b = Backward(M, N, K, dtype, "gelu", pad=pad)
        b.run()
        b.check(what)


@pytest.mark.parametrize("M,N,K", HUGE)
def test_linear_backward_more_tiles_than_cus(M, N, K):
    require_gpu()
    b = Backward(M, N, K, "f16", "none", "f32", accumulate=True)
    log(f"linear_backward {M}x{N}x{K}")
    b.run()
    b.check(f"linear_backward {M}x{N}x{K}")


def test_linear_backward_each_gradient_alone():
    require_gpu()
    for keep in ("dx", "dw", "db"):
        b = Backward(90, 130, 70, "bf16", "silu")
        over = {k: None for k in ("dx", "dw", "db") if k != keep}
        if keep != "dw":
            over["x"] = None
        if keep != "dx":
            over["w"] = None
        log(f"linear_backward {keep} alone")
        b.run(**over)
        torch.cuda.synchronize()
        wants, bounds = b.bounds()
        i = ("dx", "dw", "db").index(keep)
        m = (b.dx, b.dw, b.db)[i]
        assert_close(m.f64() if i < 2 else m.f64()[0], wants[i], bounds[i], keep)
        for other in {"dx": (b.dw, b.db), "dw": (b.dx, b.db), "db": (b.dx, b.dw)}[keep]:
            assert torch.isnan(other.buffer).all()


def test_linear_backward_of_no_rows_and_no_columns():
    require_gpu()
    log("linear_backward M = 0")
    b = Backward(0, 40, 50, "f16", "relu")
    b.run()
    torch.cuda.synchronize()
    assert (b.dw.f64() == 0).all() and (b.db.f64() == 0).all()
    log("linear_backward M = 0, accumulate")
    b = Backward(0, 40, 50, "f16", "relu", "f32", True)
    b.run()
    torch.cuda.synchronize()
    assert np.array_equal(b.dw.f64(), b.dw0) and np.array_equal(b.db.f64(), b.db0)
    log("linear_backward N = 0")
    b = Backward(60, 0, 50, "f16")
    b.run()
    torch.cuda.synchronize()
    assert (b.dx.f64() == 0).all()


def test_linear_backward_on_another_stream_twice_the_same():
    require_gpu()
    b = Backward(513, 264, 520, "bf16", "gelu")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    log("linear_backward on a side stream")
    b.run(stream=side)
    b.check("linear_backward, side stream")
    first = [m.buffer.clone() for m in (b.dx, b.dw, b.db)]
    b.run(stream=side)
    torch.cuda.synchronize()
    for was, m in zip(first, (b.dx, b.dw, b.db)):
        assert torch.equal(was.view(torch.int16), m.buffer.view(torch.int16))


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_is_the_forward_oracles_slope(act):
    """The kernel's gradients against central differences of the forward definition, along random directions."""
    require_gpu()
    b = Backward(40, 72, 48, "f16", act)
    # z belongs to x and w here, so that the loss sum(dy * y) has these gradients
    x, w = b.x.f64(), b.w.f64()
    if b.z is not None:
        b.z.view.copy_(torch.from_numpy(x @ w.T))
    log(f"linear_backward against differences, {act}")
    b.run()
    torch.cuda.synchronize()
    dy = b.dy.f64()
    z = b.z.f64() if b.z else x @ w.T
    g = np.random.default_rng(5)
    h = 1e-4
    _, bounds = b.bounds()
    for name, got, bound, along in (("dx", b.dx.f64(), bounds[0], lambda d, s: ((z + s * h * (d @ w.T)))),
                                    ("dw", b.dw.f64(), bounds[1], lambda d, s: (z + s * h * (x @ d.T)))):
        d = g.standard_normal(got.shape)
        lo, hi = along(d, -1), along(d, 1)
        diff = ((act_oracle(hi, act) - act_oracle(lo, act)) * dy).sum() / (2 * h)
        # where a relu's kink lies between the two points the difference is no slope: leave those out of both
        crossed = (np.sign(hi) != np.sign(lo)) if act == "relu" else np.zeros_like(z, bool)
        diff -= ((act_oracle(hi, act) - act_oracle(lo, act)) * dy * crossed).sum() / (2 * h)
        inner = (hi - lo) / (2 * h)
        skipped = (slope_oracle(z, act) * dy * crossed * inner).sum()
        # third derivatives of the activations are below 3: h^2/6 of it, per element
        bend = (np.abs(dy) * np.abs(inner) ** 3).sum() * h * h / 2
        # cancellation in the difference
        round64 = 1e-12 * (np.abs(act_oracle(z, act)) * np.abs(dy)).sum() / h
        assert abs((got * d).sum() - (diff + skipped)) <= (bound * np.abs(d)).sum() + bend + round64, name


# ------------------------------------------------------------------ capture

def test_linear_and_backward_captured_and_replayed():
    require_gpu()
    f = Forward(300, 264, 1100, "bf16", "gelu")
    b = Backward(300, 264, 1100, "bf16", "gelu", "f32", accumulate=False)
    fa, ba = f.args(), b.args()
    ws = workspace(ag.plan_linear(**fa)), workspace(ag.plan_linear_backward(**ba))

    def calls(stream):
        ag.linear(**fa, workspace=ws[0], stream=stream)
        ag.linear_backward(**ba, workspace=ws[1], stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for rep in range(3):
        for m, s in ((f.x, 100), (f.w, 200), (b.dy, 300), (b.z, 400)):
            g = np.random.default_rng([s, rep])
            m.view.copy_(torch.from_numpy(g.standard_normal((m.rows, m.cols)) * (0.03 if m is f.w else 1.0)).to(TORCH[m.dtype]))
        torch.cuda.synchronize()
        log(f"linear graph replay {rep}")
        graph.replay()
        f.check(f"linear, replay {rep}")
        b.check(f"linear_backward, replay {rep}")


def test_half_steps():
    assert HALF_STEP == {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
