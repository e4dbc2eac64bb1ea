"""Activations and their slopes at pre-activations up to the type's largest and lowest values.

There they are their limits: the argument or 0, and a slope of 1 or 0.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from tests.gpu_util import log, require_gpu
from tests.linear_util import TORCH

pytestmark = pytest.mark.gpu

ACTS = ["relu", "gelu", "gelu_tanh", "silu"]
LARGE_ARGUMENTS = {"bf16": [1e3, 1e9, 1.8e19, 1.9e19, 1e20, 1e30, 3.3e38, torch.finfo(torch.bfloat16).max],
                   "f16": [200.0, 1e3, 3e4, 65504.0]}


def pre_activations(dtype):
    v = LARGE_ARGUMENTS[dtype]
    z = torch.tensor(v + [-x for x in v], dtype=torch.float64).to(TORCH[dtype])
    return z.repeat(5)[:64 + len(v)].contiguous()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 40])
def test_activation_at_large_arguments(M, act, dtype):
    require_gpu()
    z = pre_activations(dtype).cuda()
    N, K = z.numel(), 32
    x, w = (torch.zeros(r, K, dtype=TORCH[dtype], device="cuda") for r in (M, N))
    y, kept = (torch.empty(M, N, dtype=TORCH[dtype], device="cuda") for _ in range(2))
    args = dict(x=x, w=w, y=y, M=M, N=N, K=K, dtype=dtype, act=act, bias=z, z=kept)
    ws = torch.empty(max(1, ag.plan_linear(**args).workspace_bytes), dtype=torch.uint8, device="cuda")
    log(f"linear at large arguments, {M} rows {act} {dtype}")
    ag.linear(**args, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(kept, z.expand(M, N))
    assert torch.equal(y.double(), torch.where(z > 0, z, torch.zeros_like(z)).double().expand(M, N))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 40])
def test_slope_at_large_arguments(M, act, dtype):
    require_gpu()
    z = pre_activations(dtype).cuda().expand(M, -1).contiguous()
    N, K = z.shape[1], 32
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    dy = torch.randn(M, N, generator=g, device="cuda").to(TORCH[dtype])
    x = torch.zeros(M, K, dtype=TORCH[dtype], device="cuda")
    x[0, 0] = 1.0                               # dw's column 0 is dz's row 0
    w = torch.zeros(N, K, dtype=TORCH[dtype], device="cuda")
    w[:K, :K] = torch.eye(K, device="cuda").to(TORCH[dtype])       # dx is dz's first columns
    dx, dw, db = torch.empty_like(x), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    args = dict(dy=dy, z=z, x=x, w=w, M=M, N=N, K=K, dtype=dtype, act=act, dx=dx, dw=dw, db=db, dw_dtype="f32")
    ws = torch.empty(max(1, ag.plan_linear_backward(**args).workspace_bytes), dtype=torch.uint8, device="cuda")
    log(f"linear_backward at large arguments, {M} rows {act} {dtype}")
    ag.linear_backward(**args, workspace=ws)
    torch.cuda.synchronize()
    dz = torch.where(z > 0, dy, torch.zeros_like(dy)).double()
    assert torch.equal(dx.double(), dz[:, :K])
    assert torch.equal(dw.double()[:, 0], dz[0]) and not dw[:, 1:].any()
    size = dy.double().abs().sum(0).cpu().numpy()
    assert (np.abs((db.double() - dz.sum(0)).cpu().numpy()) <= (M + 8) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("act", ACTS)
def test_slope_of_nan_is_nan_but_for_relu(act):
    """A NaN pre-activation makes its own gradient NaN (relu's comparison lets dy through) and no other one."""
    require_gpu()
    z = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    z[0, 9] = float("nan")
    dy = torch.ones_like(z)
    db = torch.empty(64, device="cuda")
    args = dict(dy=dy, z=z, x=None, w=None, M=1, N=64, K=8, dtype="bf16", act=act, db=db, dw_dtype="f32")
    ws = torch.empty(max(1, ag.plan_linear_backward(**args).workspace_bytes), dtype=torch.uint8, device="cuda")
    log(f"linear_backward with a NaN, {act}")
    ag.linear_backward(**args, workspace=ws)
    torch.cuda.synchronize()
    nan = torch.isnan(db)
    assert not nan[torch.arange(64) != 9].any() and bool(nan[9]) == (act != "relu")
