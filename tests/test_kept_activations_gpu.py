"""The operators on 8-bit rows as they are used together: a block's serving and training, against the same in float64.

Serving: the residual's addition and the norm with 8-bit output, the layer on 8-bit integers.  Training: the norm, the layer,
its input and pre-activation kept in 8 bits, then the gradients back through the layer and the norm.  Codes come from the
kernels (they have to match the oracle's exactly); every later step's reference starts from what the step before stored.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import act_oracle, linear_backward_oracle
from oracle.rows_oracle import codes_product_oracle, norm_backward_oracle, norm_oracle, quantize_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import ACT_ERROR, HALF_STEP, TINY, TORCH, U32, assert_close, product_bound, rounded_bound
from tests.rows_util import activations, assert_codes

pytestmark = pytest.mark.gpu

EPS = 1e-5


def f64(t):
    return t.double().cpu().numpy()


def room(*plans):
    return torch.full((max([1] + [p.workspace_bytes for p in plans]),), 0xA5, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 13, 300])
def test_serving(M, dtype):
    """One token, a few, a prompt: x + residual, norm, codes, layer with bias, activation and the residual stream."""
    require_gpu()
    log(f"serving {M} rows {dtype}")
    K, N = 1032, 520
    g = np.random.default_rng(M)
    dev = lambda a: torch.as_tensor(a).to(TORCH[dtype]).cuda()  # noqa: E731
    x, r = activations(1, M, K, dtype).cuda(), activations(2, M, K, dtype).cuda()
    norm, w, b = dev(1 + 0.1 * g.standard_normal(K)), dev(g.standard_normal((N, K)) / np.sqrt(K)), dev(g.standard_normal(N))
    skip = dev(g.standard_normal((M, N)))
    wq, ws = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    h, y = torch.empty_like(x), torch.empty(M, N, dtype=TORCH[dtype], device="cuda")
    ag.quantize_rows(w, wq, ws, N, K, dtype)                # once, when the weights are loaded
    space = room(ag.plan_linear_i8(q, wq, s, ws, y, M, N, K, dtype, "silu", b, skip))
    ag.rms_norm(x, M, K, dtype, norm, r, h, q=q, scale=s, eps=EPS)
    ag.linear_i8(q, wq, s, ws, y, M, N, K, dtype, "silu", b, skip, workspace=space)
    torch.cuda.synchronize()
    assert torch.equal(h.cpu(), (x.double() + r.double()).to(TORCH[dtype]).cpu())
    _, _, codes, scale = norm_oracle(f64(h), f64(norm), EPS)
    wcodes, wscale = quantize_oracle(f64(w))
    assert_codes(q.cpu().numpy(), codes, "codes of x")
    assert_codes(wq.cpu().numpy(), wcodes, "codes of w")
    assert_close(f64(s), scale, 3.6 * U32 * scale, "scale of x")
    assert_close(f64(ws), wscale, U32 * (1 + 2.0 ** -20) * wscale, "scale of w")
    p = codes_product_oracle(codes, wcodes, f64(s), f64(ws))
    z = p + f64(b)
    want = act_oracle(z, "silu") + f64(skip)
    off = 1.13 * (3.01 * U32 * np.abs(p) + U32 * (np.abs(z) + np.abs(f64(b)))) + ACT_ERROR * np.abs(z) + U32 * (np.abs(want) + np.abs(f64(skip)))
    assert_close(f64(y), want, rounded_bound(want, off, dtype), "y")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_training(dtype):
    """Forward with what the backward pass needs kept in 8 bits; the gradients of the layer and, through them, of the norm."""
    require_gpu()
    log(f"training {dtype}")
    M, K, N = 260, 520, 392
    g = np.random.default_rng(7)
    dev = lambda a: torch.as_tensor(a).to(TORCH[dtype]).cuda()  # noqa: E731
    new = lambda *shape, t=TORCH[dtype]: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
    x, r = activations(1, M, K, dtype).cuda(), activations(2, M, K, dtype).cuda()
    norm, w, b = dev(1 + 0.1 * g.standard_normal(K)), dev(g.standard_normal((N, K)) / np.sqrt(K)), dev(g.standard_normal(N))
    dy, dh = dev(g.standard_normal((M, N))), dev(g.standard_normal((M, K)))
    h, n, rstd, y, z = new(M, K), new(M, K), new(M, t=torch.float32), new(M, N), new(M, N)
    n8, ns, z8, zs = new(M, K, t=torch.int8), new(M, t=torch.float32), new(M, N, t=torch.int8), new(M, t=torch.float32)
    dn, dw, db, dx, dnorm = new(M, K), new(N, K, t=torch.float32), new(N, t=torch.float32), new(M, K), new(K, t=torch.float32)
    back = dict(dy=dy, x=n8, x_scale=ns, w=w, M=M, N=N, K=K, dtype=dtype, act="gelu", z=z8, z_scale=zs, dx=dn, dw=dw, db=db, dw_dtype="f32")
    norm_back = dict(dy=dn, h=h, rstd=rstd, M=M, K=K, dtype=dtype, weight=norm, dh=dh, dx=dx, dw=dnorm, dw_dtype="f32")
    space = room(ag.plan_linear(n, w, y, M, N, K, dtype, "gelu", b, z=z), ag.plan_linear_backward_q8(**back),
                 ag.plan_rms_norm_backward(**norm_back))
    ag.rms_norm(x, M, K, dtype, norm, r, h, n, rstd=rstd, eps=EPS)
    ag.linear(n, w, y, M, N, K, dtype, "gelu", b, z=z, workspace=space)
    ag.quantize_rows(n, n8, ns, M, K, dtype)
    ag.quantize_rows(z, z8, zs, M, N, dtype)
    n16 = n.clone()
    n.fill_(float("nan")), z.fill_(float("nan"))            # the backward pass has the codes alone
    ag.linear_backward_q8(**back, workspace=space)
    ag.rms_norm_backward(**norm_back, workspace=space)      # the same workspace: the calls are in order on one stream
    torch.cuda.synchronize()
    want_n = norm_oracle(f64(h), f64(norm), EPS)[0]
    assert_close(f64(n16), want_n, rounded_bound(want_n, 3.6 * U32 * np.abs(want_n), dtype), "norm")
    codes, _ = quantize_oracle(f64(n16))
    assert_codes(n8.cpu().numpy(), codes, "kept norm")
    nk, zk = codes * f64(ns)[:, None], z8.cpu().numpy() * f64(zs)[:, None]
    want_dn, want_dw, want_db, dz = linear_backward_oracle(f64(dy), zk, nk, f64(w), "gelu")
    # dz's evaluation and, for dn, its rounding; for dw two terms (bf16: three) of dz times a factor of at least 1/2
    half, tiny = HALF_STEP[dtype], TINY[dtype]
    dz_off = (ACT_ERROR * (1 + np.abs(zk)) + U32 + 1.2 * U32 * np.abs(zk)) * np.abs(f64(dy))
    dz_x = rounded_bound(dz, dz_off, dtype)
    off = dz_x @ np.abs(f64(w)) + product_bound(np.abs(dz) + dz_x, f64(w).T, N)
    assert_close(f64(dn), want_dn, rounded_bound(want_dn, off, dtype), "gradient of the layer's input")
    folded = dz_off + U32 * np.abs(dz)
    dz_w = half * (np.abs(dz) + folded) + 2 * tiny
    for _ in range(2 if dtype == "bf16" else 1):
        dz_w = half * dz_w + 2 * tiny
    dz_w = folded + dz_w
    off = dz_w.T @ np.abs(nk) + 3 * product_bound((np.abs(dz) + dz_w).T, nk.T, M + 2)
    assert_close(f64(dw), want_dw, rounded_bound(want_dw, off, "f32"), "gradient of the weight")
    assert_close(f64(db), want_db, rounded_bound(want_db, dz_off.sum(0) + (M + 8) * U32 * (np.abs(dz) + dz_off).sum(0), "f32"), "gradient of the bias")
    # the norm's, from the gradient that was stored
    d, hh, rr, ww = f64(dn), f64(h), f64(rstd), f64(norm)
    want_dx, want_dnorm = norm_backward_oracle(d, hh, rr, ww, f64(dh))
    nn, gg = hh * rr[:, None], d * ww
    c = np.abs((gg * nn).sum(1) / K)[:, None]
    c_off = 60 * U32 * np.abs(gg * nn).sum(1)[:, None] / K
    off = rr[:, None] * ((np.abs(gg) + np.abs(nn) * c) * 4 * U32 + np.abs(nn) * c_off) + U32 * np.abs(want_dx)
    assert_close(f64(dx), want_dx, rounded_bound(want_dx, off, dtype), "gradient of x and the residual")
    assert_close(f64(dnorm), want_dnorm, (M + 40) * U32 * np.abs(d * nn).sum(0) + TINY["f32"], "gradient of the norm's weight")
