"""The linear layer on 8-bit integers on the GPU against exact sums.

The integer sums are exact, so the bounds hold the epilogue alone: three fp32 roundings for the sum's conversion and the
two scales, then bias, activation, residual and the one rounding as in the 16-bit layer.  Operands of codes lie among other
codes, outputs in NaN, at odd strides and offsets.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import act_oracle
from oracle.rows_oracle import codes_product_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import ACT_ERROR, HUGE, LARGE, U32, Matrix, assert_close, random_matrix, rounded_bound
from tests.rows_util import CodeMatrix, vector
from tests.test_linear_gpu import ACTS, SIZES, workspace

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, M, N, K, dtype, act="none", bias=True, residual=True, z=True, pad=0, offset=0, seed=1, lowest=-127):
        self.shape, self.dtype, self.act = (M, N, K), dtype, act
        g = np.random.default_rng([seed, M, N, K])
        codes = lambda *s: g.integers(lowest, 128, s, dtype=np.int8)  # noqa: E731
        self.x = CodeMatrix(M, K, pad, offset, codes(M, K))
        self.w = CodeMatrix(N, K, pad, offset, codes(N, K))
        # sums of about sqrt(K) 74^2 become about 1
        self.xs = vector(M, offset, np.exp(g.standard_normal(M)) / 74)
        self.ws = vector(N, offset, np.exp(0.3 * g.standard_normal(N)) / 74 / np.sqrt(max(K, 1)))
        self.b = random_matrix(seed + 2, 1, N, dtype, 0.5, offset=offset) if bias else None
        self.r = random_matrix(seed + 3, M, N, dtype, pad=pad, offset=offset) if residual else None
        self.y = Matrix(M, N, dtype, pad=pad, offset=offset)
        self.z = Matrix(M, N, dtype, pad=pad, offset=offset) if z else None

    def args(self):
        M, N, K = self.shape
        at = lambda m: m.ptr if m is not None else None  # noqa: E731
        ld = lambda m: m.ld if m is not None else 0  # noqa: E731
        return dict(x=self.x.ptr, w=self.w.ptr, x_scale=self.xs.ptr, w_scale=self.ws.ptr, y=self.y.ptr, M=M, N=N, K=K,
                    dtype=self.dtype, act=self.act, bias=at(self.b), residual=at(self.r), z=at(self.z), ldx=self.x.ld, ldw=self.w.ld,
                    ldr=ld(self.r), ldy=self.y.ld, ldz=ld(self.z))

    def run(self, stream=None):
        a = self.args()
        ag.linear_i8(**a, workspace=workspace(ag.plan_linear_i8(**a)), stream=stream)

    def check(self, what, residual=None):
        torch.cuda.synchronize()
        p = codes_product_oracle(self.x.numpy(), self.w.numpy(), self.xs.f64()[0], self.ws.f64()[0])
        b = self.b.f64() if self.b is not None else 0.0
        z = p + b
        r = residual if residual is not None else self.r.f64() if self.r is not None else 0.0
        y = act_oracle(z, self.act) + r
        off = 3.01 * U32 * np.abs(p) + U32 * (np.abs(z) + np.abs(b))
        if self.z is not None:
            assert_close(self.z.f64(), z, rounded_bound(z, off, self.dtype), what + " z")
            self.z.check_surroundings(what + " z")
        # no slope is above 1.13
        off = 1.13 * off + ACT_ERROR * np.abs(z) + U32 * (np.abs(y) + np.abs(r))
        assert_close(self.y.f64(), y, rounded_bound(y, off, self.dtype), what + " y")
        self.y.check_surroundings(what + " y")
        for m in (self.x, self.w):
            m.check_surroundings(what)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_i8_sizes(M, N, K, dtype):
    require_gpu()
    for i, (pad, offset) in enumerate([(0, 0), (16, 0), (4, 4), (3, 1), (6, 2), (5, 0)]):
        act = ACTS[(i + M + N) % 5]
        what = f"linear_i8 {M}x{N}x{K} {dtype} {act} pad {pad} offset {offset}"
        log(what)
        f = Layer(M, N, K, dtype, act, pad=pad, offset=offset, seed=10 * i)
        f.run()
        f.check(what)


@pytest.mark.parametrize("M,K", [(5, 255), (5, 256), (5, 257), (16, 4097), (20, 513), (70, 127), (70, 128), (70, 129), (70, 1),
                                 (130, 255), (130, 383), (300, 641)])
def test_linear_i8_ends_of_the_reduction(M, K):
    """Rows that end inside a stage, a 16-byte vector or a word, with other codes right behind them."""
    require_gpu()
    for pad, offset in ((0, 0), (1, 3), (4, 0)):
        what = f"linear_i8 {M}x130x{K} pad {pad} offset {offset}"
        log(what)
        f = Layer(M, 130, K, "bf16", pad=pad, offset=offset)
        f.run()
        f.check(what)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 70])
def test_linear_i8_epilogue_parts(M, act):
    require_gpu()
    for bias in (False, True):
        for residual in (False, True):
            for z in (False, True):
                what = f"linear_i8 {M} {act} bias {bias} residual {residual} z {z}"
                log(what)
                f = Layer(M, 200, 96, "bf16", act, bias, residual, z, pad=4)
                f.run()
                f.check(what)


@pytest.mark.parametrize("M,N,K", LARGE + [(700, 700, 20000), (300, 264, 16001)])
def test_linear_i8_larger_sizes(M, N, K):
    require_gpu()
    for i, (dtype, pad) in enumerate((("f16", 0), ("bf16", 12), ("bf16", 1))):
        what = f"linear_i8 {M}x{N}x{K} {dtype} pad {pad}"
        log(what)
        f = Layer(M, N, K, dtype, ACTS[i + 2], pad=pad)
        p = ag.plan_linear_i8(**f.args()).product
        log(f"  tile {p.tile_m}x{p.tile_n} full {p.full_tiles} of {p.n_programs} programs, splits {p.splits} packed {p.packed}")
        f.run()
        f.check(what)


@pytest.mark.parametrize("i", [0, 2])
def test_linear_i8_more_tiles_than_cus(i):
    require_gpu()
    M, N, K = HUGE[i]
    f = Layer(M, N, K, "bf16", "silu", z=False)
    p = ag.plan_linear_i8(**f.args()).product
    log(f"linear_i8 {M}x{N}x{K}: tile {p.tile_m}x{p.tile_n} full {p.full_tiles} splits {p.splits}")
    f.run()
    f.check(f"linear_i8 {M}x{N}x{K}")


@pytest.mark.parametrize("M", [2, 40])
def test_linear_i8_largest_sums(M):
    """K at its limit and codes of -128 everywhere: the sums reach 2^31 - 2^14."""
    require_gpu()
    N, K = 24, 131071
    log(f"linear_i8 {M}x{N}x{K} of -128")
    f = Layer(M, N, K, "bf16")
    f.x.view.fill_(-128)
    f.w.view.fill_(-128)
    f.w.view[3].fill_(127)
    f.x.snapshot(), f.w.snapshot()
    f.run()
    f.check(f"linear_i8 {M}x{N}x{K}")


@pytest.mark.parametrize("M", [0, 1, 40])
def test_linear_i8_without_reduction_or_output(M):
    """K = 0 leaves act(bias) + residual; M = 0 or N = 0 nothing to do."""
    require_gpu()
    for N, K in ((24, 0), (0, 24), (0, 0)):
        log(f"linear_i8 {M}x{N}x{K}")
        f = Layer(M, N, K, "f16", "silu")
        f.run()
        f.check(f"linear_i8 {M}x{N}x{K}")


@pytest.mark.parametrize("M", [3, 300])
def test_linear_i8_residual_in_place(M):
    require_gpu()
    log(f"linear_i8 {M}: y is the residual")
    f = Layer(M, 136, 264, "bf16", "gelu", z=False)
    r = f.r.f64()
    f.y = f.r
    f.run()
    f.check(f"linear_i8 {M} in place", residual=r)


@pytest.mark.parametrize("M", [3, 90, 520])
def test_linear_i8_scales_of_nan_and_zero(M):
    """A row or channel whose scale is NaN (it held one) is NaN, one whose scale is 0 is the bias's."""
    require_gpu()
    log(f"linear_i8 {M}: NaN and zero scales")
    f = Layer(M, 140, 300, "bf16", residual=False, z=False)
    f.xs.view[0, 1], f.xs.view[0, 2], f.ws.view[0, 7] = float("nan"), 0.0, float("nan")
    f.run()
    torch.cuda.synchronize()
    y = f.y.f64()
    assert np.isnan(y[1]).all() and np.isnan(y[:, 7]).all()
    others = np.delete(np.arange(140), 7)
    assert np.array_equal(y[2, others], f.b.f64()[0, others])
    assert np.isfinite(np.delete(np.delete(y, 1, 0), 7, 1)).all()


def test_linear_i8_extreme_scales():
    """Scales whose product leaves fp32 though the result does not."""
    require_gpu()
    for M in (3, 90):
        log(f"linear_i8 {M}: extreme scales")
        f = Layer(M, 70, 64, "bf16", bias=False, residual=False, z=False)
        f.xs.view.fill_(2.0 ** -100)
        f.ws.view.fill_(2.0 ** 90)
        f.run()
        f.check(f"linear_i8 {M} extreme scales")


def test_linear_i8_offsets_past_32_bits():
    """Rows of x, w, y and z that lie past 2^32 bytes."""
    require_gpu()
    M, N, K, ld = 4200, 2100, 64, 1 << 20
    log(f"linear_i8 {M}x{N}x{K} at stride {ld}")
    g = np.random.default_rng(3)
    wide = lambda rows, cols, dtype: torch.zeros((rows - 1) * ld + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (ld, 1))  # noqa: E731
    x, w, y = wide(M, K, torch.int8), wide(N, K, torch.int8), wide(M, N, torch.bfloat16)
    x0, w0 = (g.integers(-127, 128, (n, K), dtype=np.int8) for n in (M, N))
    x.copy_(torch.from_numpy(x0)), w.copy_(torch.from_numpy(w0))
    xs, ws = np.full(M, 0.01, np.float32), np.full(N, 0.01, np.float32)
    a = dict(x=x, w=w, x_scale=torch.from_numpy(xs).cuda(), w_scale=torch.from_numpy(ws).cuda(), y=y, M=M, N=N, K=K, dtype="bf16",
             ldx=ld, ldw=ld, ldy=ld)
    ag.linear_i8(**a, workspace=workspace(ag.plan_linear_i8(**a)))
    torch.cuda.synchronize()
    want = codes_product_oracle(x0, w0, xs, ws)
    assert_close(y.double().cpu().numpy(), want, rounded_bound(want, 3.01 * U32 * np.abs(want), "bf16"), "y")


def test_linear_i8_stays_inside_its_workspace():
    """On another stream than the current one, between guards, twice with the same bits."""
    require_gpu()
    side, guard = torch.cuda.Stream(), 1 << 16
    for M, N, K, pad in ((33, 600, 8200, 0), (700, 700, 16384, 0), (300, 264, 2200, 3), (513, 520, 4099, 1)):
        f = Layer(M, N, K, "bf16", "gelu", pad=pad)
        need = ag.plan_linear_i8(**f.args()).workspace_bytes
        assert need
        ws = torch.full((need + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
        first = None
        for _ in range(2):
            ws[guard:guard + need] = 0xFF
            side.wait_stream(torch.cuda.current_stream())
            log(f"linear_i8 {M}x{N}x{K} on a side stream")
            ag.linear_i8(**f.args(), workspace=ws[guard:guard + need], stream=side)
            torch.cuda.synchronize()
            f.check(f"linear_i8 {M}x{N}x{K}")
            assert bool((ws[:guard] == 0x5A).all()) and bool((ws[guard + need:] == 0x5A).all())
            bits = [m.buffer.view(torch.int16).clone() for m in (f.y, f.z)]
            assert first is None or all(torch.equal(u, v) for u, v in zip(first, bits))
            first = bits


def test_norm_and_linear_i8_in_a_graph():
    """The norm's codes into the layer, one token and many, captured once and replayed on new inputs."""
    require_gpu()
    for M in (1, 200):
        log(f"norm and linear_i8 in a graph, {M} rows")
        N, K = 520, 1000
        g = torch.Generator(device="cuda").manual_seed(M)
        x, r, h = (torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        w = torch.randn(N, K, generator=g, device="cuda").bfloat16()
        norm = torch.ones(K, dtype=torch.bfloat16, device="cuda")
        q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        wq, ws = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        ag.quantize_rows(w, wq, ws, N, K, "bf16")
        space = torch.empty(max(1, ag.plan_linear_i8(q, wq, s, ws, y, M, N, K, "bf16").workspace_bytes), dtype=torch.uint8, device="cuda")

        def step(stream):
            ag.rms_norm(x, M, K, "bf16", norm, r, h, q=q, scale=s, stream=stream)
            ag.linear_i8(q, wq, s, ws, y, M, N, K, "bf16", workspace=space, stream=stream)

        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        x.normal_(generator=g), r.normal_(generator=g)
        torch.cuda.synchronize()
        step(side)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step(side)
        for i in range(4):
            x.normal_(generator=g), r.normal_(generator=g)
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (h, q, s, y)]
            step(torch.cuda.current_stream())
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(got, (h, q, s, y))), f"replay {i}"
            # the whole way against the layer of the unquantized rows: 8 bits leave about a percent
            want = (h.double() / (h.double().square().mean(1, keepdim=True) + 1e-6).sqrt()) @ w.double().t()
            assert float((y.double() - want).norm() / want.norm()) < 0.03
