"""Weight gradients asked for in fp32 behind an activation: dz may not leave its 16-bit rounding in them.

The bound is that of two 16-bit terms: what the first one leaves (half a step of dz) is itself rounded by half a
step, so dz is off by the square of a half step, beside its evaluation in fp32.
"""

import pytest
import torch

import numpy as np

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import linear_backward_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import ACT_ERROR, HALF_STEP, TINY, U32, assert_close, rounded_bound
from tests.test_linear_gpu import Backward

pytestmark = pytest.mark.gpu

# gradients side by side, in turn, apart and cut; one row, a ragged reduction, rows to be copied first
SHAPES = [(1, 40, 24, 0), (33, 65, 70, 0), (150, 264, 200, 0), (150, 264, 200, 3), (700, 700, 2100, 0), (1000, 1030, 2050, 8),
          (8300, 1100, 600, 0)]


def check_dw(b, what):
    M, N, K = b.shape
    dy, x, w, z = b.dy.f64(), b.x.f64(), b.w.f64(), b.z.f64()
    _, dw, _, dz = linear_backward_oracle(dy, z, x, w, b.act)
    h, tiny = HALF_STEP[b.dtype], TINY[b.dtype]
    evaluated = (ACT_ERROR * (1 + np.abs(z)) + U32) * np.abs(dy)
    off_dz = evaluated + h * (h * (np.abs(dz) + evaluated) + tiny) + tiny
    size = (np.abs(dz) + off_dz).T @ np.abs(x)
    # two fp32 sums, the second added to the first's result
    off = off_dz.T @ np.abs(x) + (2 * (M + 8) + 2) * U32 * size
    if b.accumulate:
        dw = dw + b.dw0
        off = off + 2 * U32 * np.abs(b.dw0)
    torch.cuda.synchronize()
    assert_close(b.dw.f64(), dw, rounded_bound(dw, off, "f32"), what)
    b.dw.check_surroundings(what)


@pytest.mark.parametrize("dtype,act", [("bf16", "gelu"), ("bf16", "silu"), ("f16", "gelu_tanh")])
@pytest.mark.parametrize("M,N,K,pad", SHAPES)
def test_fp32_weight_gradient_behind_an_activation(M, N, K, pad, dtype, act):
    require_gpu()
    for accumulate in (False, True):
        what = f"linear_backward {M}x{N}x{K} {dtype} {act} pad {pad} dw f32 accumulate {accumulate}"
        log(what)
        b = Backward(M, N, K, dtype, act, "f32", accumulate, pad=pad, seed=3)
        b.run()
        check_dw(b, what)
        b.check(what)       # dx and db too, to the bounds of every gradient


def test_fp32_weight_gradient_alone():
    require_gpu()
    b = Backward(90, 130, 70, "bf16", "silu", "f32")
    log("linear_backward dw f32 alone")
    b.run(dx=None, db=None, w=None)
    check_dw(b, "dw alone")
    assert torch.isnan(b.dx.buffer).all() and torch.isnan(b.db.buffer).all()


def test_overflow_of_dz_stays_infinite():
    """dz past fp16's largest value is an infinity in the products, with no NaN from what it leaves."""
    require_gpu()
    b = Backward(40, 24, 16, "f16", "gelu", "f32")
    b.z.view.fill_(1.5)                 # the slope's largest region: above 1.12
    b.dy.view.fill_(1.0)
    b.dy.view[3, 5] = 65504.0
    b.x.view.fill_(1.0)
    log("linear_backward with dz past fp16")
    b.run()
    torch.cuda.synchronize()
    dw = b.dw.f64()
    assert np.isposinf(dw[5]).all() and np.isfinite(np.delete(dw, 5, 0)).all()


@pytest.mark.parametrize("M,N,K", [(300, 264, 1100), (2048, 520, 264)])
def test_fp32_weight_gradient_captured_and_replayed(M, N, K):
    require_gpu()
    b = Backward(M, N, K, "bf16", "gelu", "f32")
    args = b.args()
    need = ag.plan_linear_backward(**args).workspace_bytes
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ag.linear_backward(**args, workspace=ws, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ag.linear_backward(**args, workspace=ws, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for rep in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(rep)
        for m in (b.dy, b.z, b.x):
            m.view.copy_(torch.randn(m.rows, m.cols, generator=g, device="cuda"))
        torch.cuda.synchronize()
        log(f"linear_backward dw f32, replay {rep}")
        graph.replay()
        check_dw(b, f"replay {rep}")
