"""More rows than a launch has workgroups (2^22 - 1): each workgroup takes several in turn, and its LDS in turn with them.

Rows repeat with a period that the workgroups' number is no multiple of, so that a row left out, taken twice or mixed with the
one before is seen; the period itself is checked against the oracle.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.rows_oracle import norm_oracle, quantize_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import TINY, TORCH, U32, assert_close
from tests.rows_util import activations, assert_codes

pytestmark = pytest.mark.gpu

GROUPS, PERIOD = (1 << 22) - 1, 61


def f64(t):
    return t.double().cpu().numpy()


def repeated(period, M):
    """M rows, the period's over and over."""
    return torch.cat([period.repeat(M // PERIOD, 1), period[:M % PERIOD]])


def assert_repeats(got, period, what):
    """got's rows are the period's over and over, bit for bit; in pieces, for the comparison's memory."""
    step = PERIOD * max(1, (1 << 28) // (PERIOD * period.shape[1]))
    for at in range(0, got.shape[0], step):
        piece = got[at:at + step]
        assert torch.equal(piece, repeated(period, piece.shape[0])), f"{what}: rows from {at} on"


@pytest.mark.parametrize("K,per_group,norm", [(16, 16, True), (136, 4, True), (1032, 1, True), (4104, 1, False)])
def test_more_rows_than_workgroups(K, per_group, norm):
    require_gpu()
    M = (GROUPS + 5) * per_group + 1
    log(f"{'norm' if norm else 'codes'} {M}x{K}")
    period = activations(K, PERIOD, K, "bf16").cuda()
    x, q, scale = repeated(period, M), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    rstd = torch.empty(M, device="cuda") if norm else None
    if norm:
        ag.rms_norm(x, M, K, "bf16", q=q, scale=scale, rstd=rstd, eps=1e-6)
        _, root, codes, sizes = norm_oracle(f64(period), None, 1e-6)
        assert_close(f64(rstd[:PERIOD]), root, 2.5 * U32 * root, "rstd")
        assert_repeats(rstd[:, None], rstd[:PERIOD, None], "rstd")
    else:
        ag.quantize_rows(x, q, scale, M, K, "bf16")
        codes, sizes = quantize_oracle(f64(period))
    torch.cuda.synchronize()
    assert_codes(q[:PERIOD].cpu().numpy(), codes, "codes")
    assert_close(f64(scale[:PERIOD]), sizes, 3.6 * U32 * sizes + TINY["f32"], "scale")
    assert_repeats(q, q[:PERIOD], "codes")
    assert_repeats(scale[:, None], scale[:PERIOD, None], "scale")
    del x, q, scale, rstd
    torch.cuda.empty_cache()


def test_more_kept_rows_than_workgroups():
    """Gradients of fp16 rows kept in 8 bits, a workgroup a row; dy is 0 but in the first and the last rows, so that the sums are short."""
    require_gpu()
    M, N, K = GROUPS + 6, 8, 2056
    log(f"linear_backward_q8 {M}x{N}x{K} f16")
    g = np.random.default_rng(3)
    rows = np.r_[0:5, M - 9:M]
    dy, x, scale = torch.zeros(M, N, dtype=TORCH["f16"], device="cuda"), torch.ones(M, K, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
    at = torch.from_numpy(rows).cuda()
    dy[at] = torch.from_numpy(g.standard_normal((len(rows), N)) * np.exp2(g.integers(-14, 6, (len(rows), 1)))).half().cuda()
    x[at] = torch.from_numpy(g.integers(-127, 128, (len(rows), K), dtype=np.int8)).cuda()
    scale[at] = torch.from_numpy(np.exp2(g.uniform(-9, 0, len(rows)))).float().cuda()
    dw = torch.empty(N, K, device="cuda")
    a = dict(dy=dy, x=x, x_scale=scale, w=None, M=M, N=N, K=K, dtype="f16", dw=dw, dw_dtype="f32")
    space = torch.empty(ag.plan_linear_backward_q8(**a).workspace_bytes, dtype=torch.uint8, device="cuda")
    ag.linear_backward_q8(**a, workspace=space)
    torch.cuda.synchronize()
    d, v = f64(dy[at]), f64(x[at]) * f64(scale[at])[:, None]
    # two terms of dz times its scale: 2^-22 of an element, or 2^-24 of its row's largest; 30 additions (zeros add nothing), in which
    # codes times less than 2^-14 count as that: the power is 2^-23 at least here, so as codes of 2^9
    off = (2.0 ** -22 + U32) * np.abs(d) + 2.0 ** -24 * np.abs(d).max(1, keepdims=True)
    counts = np.maximum(np.abs(v), 2.0 ** 9 * f64(scale[at])[:, None])
    assert_close(f64(dw), d.T @ v, off.T @ np.abs(v) + 30 * U32 * (np.abs(d).T @ counts), "dw")
    del dy, x, scale, space
    torch.cuda.empty_cache()
