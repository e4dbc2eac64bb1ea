"""The erf form of gelu and its slope in the left tail, relative to their own (small) values.

The bound: exp(-z^2/2) is a power of two whose exponent takes three roundings, so it is off by 3 z^2/2 half steps of
fp32; the polynomial beside it and the few operations around them stay within 2^-18.
"""

import math

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from tests.gpu_util import log, require_gpu
from tests.linear_util import HALF_STEP, TORCH, U32, assert_close, rounded_bound

pytestmark = pytest.mark.gpu

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def arguments(dtype):
    """Every value of the type in [-12, -1/16] (fp16: its gelu is subnormal below about -4.5), whole and in between."""
    z = torch.linspace(-12.0, -1 / 16, 6000, dtype=torch.float64).to(TORCH[dtype]).unique()
    return z[: z.numel() // 8 * 8]


def relative(z):
    return 1.5 * z * z * U32 + 2.0 ** -18


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 40])
def test_gelu_in_the_left_tail(M, dtype):
    require_gpu()
    bias = arguments(dtype).cuda()
    N, K = bias.numel(), 32
    x, w = (torch.zeros(r, K, dtype=TORCH[dtype], device="cuda") for r in (M, N))
    y = torch.empty(M, N, dtype=TORCH[dtype], device="cuda")
    args = dict(x=x, w=w, y=y, M=M, N=N, K=K, dtype=dtype, act="gelu", bias=bias)
    ws = torch.empty(max(1, ag.plan_linear(**args).workspace_bytes), dtype=torch.uint8, device="cuda")
    log(f"gelu in the left tail, {M} rows {dtype}")
    ag.linear(**args, workspace=ws)
    torch.cuda.synchronize()
    z = bias.double().cpu().numpy()
    want = 0.5 * z * _erfc(-z / math.sqrt(2.0))
    bound = rounded_bound(want, relative(z) * np.abs(want), dtype)
    for row in (0, M - 1):
        assert_close(y[row].double().cpu().numpy(), want, bound, f"row {row}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gelu_slope_in_the_left_tail(dtype):
    """One row and dy = 1: db in fp32 is the slope itself."""
    require_gpu()
    z = arguments(dtype).cuda().view(1, -1)
    N = z.numel()
    dy, db = torch.ones_like(z), torch.empty(N, device="cuda")
    args = dict(dy=dy, z=z, x=None, w=None, M=1, N=N, K=8, dtype=dtype, act="gelu", db=db, dw_dtype="f32")
    ws = torch.empty(max(1, ag.plan_linear_backward(**args).workspace_bytes), dtype=torch.uint8, device="cuda")
    log(f"gelu's slope in the left tail, {dtype}")
    ag.linear_backward(**args, workspace=ws)
    torch.cuda.synchronize()
    t = z[0].double().cpu().numpy()
    whole, part = 0.5 * _erfc(-t / math.sqrt(2.0)), t * np.exp(-t * t / 2) / math.sqrt(2 * math.pi)
    # the two terms have opposite signs: each is off by its own size
    bound = relative(t) * (np.abs(whole) + np.abs(part))
    assert_close(db.double().cpu().numpy(), whole + part, rounded_bound(whole + part, bound, "f32"), "slope")


def test_half_steps_of_the_tail():
    assert HALF_STEP["bf16"] == 2.0 ** -8 and HALF_STEP["f16"] == 2.0 ** -11
