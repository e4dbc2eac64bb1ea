"""Refusals and plans of the row operators (codes of 8 bits, the root-mean-square norm and its gradients) without a GPU, and
the pins of their oracle."""

import ctypes
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor
from fractions import Fraction

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.rows_oracle import codes_product_oracle, norm_backward_oracle, norm_oracle, quantize_oracle
from tests.test_linear_cpu import A, GIB, INVALID, UNSUPPORTED, status_of

NORM = dict(x=A, M=1000, K=8192, dtype="bf16", weight=A + GIB, residual=A + 2 * GIB, h=A + 3 * GIB, y=A + 4 * GIB, q=A + 5 * GIB,
            scale=A + 6 * GIB, rstd=A + 7 * GIB, num_cus=256)
BACKWARD = dict(dy=A, h=A + GIB, rstd=A + 2 * GIB, M=1000, K=8192, dtype="f16", weight=A + 3 * GIB, dh=A + 4 * GIB, dx=A + 5 * GIB,
                dw=A + 6 * GIB, num_cus=256)
ROWS = dict(x=A, q=A + GIB, scale=A + 2 * GIB, M=100, K=4096, dtype="bf16")
VALUES = dict(q=A, scale=A + GIB, y=A + 2 * GIB, M=100, K=4096, dtype="f32")


@pytest.mark.parametrize("over,status", [
    (dict(x=None), INVALID), (dict(x=A + 1), INVALID), (dict(weight=A + GIB + 1), INVALID), (dict(scale=A + 6 * GIB + 2), INVALID),
    (dict(rstd=A + 7 * GIB + 1), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID),
    (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(M=1 << 31), UNSUPPORTED), (dict(K=(1 << 20) + 1), UNSUPPORTED),
    (dict(dtype="f32"), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=9e-61), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(ldx=8191), INVALID), (dict(ldr=1), INVALID), (dict(ldh=-1), INVALID), (dict(ldy=8000), INVALID), (dict(ldq=8191), INVALID),
    (dict(ldq=(1 << 20) + 1), UNSUPPORTED),
    (dict(y=A), INVALID), (dict(y=A + 2 * GIB), INVALID), (dict(q=A + 64), INVALID), (dict(scale=A + GIB), INVALID),
    (dict(rstd=A + 6 * GIB + 100), INVALID), (dict(h=A + 2), INVALID), (dict(h=A, ldh=9000), INVALID), (dict(h=A + GIB), INVALID),
    (dict(h=A + 4 * GIB + 16), INVALID), (dict(h=A + 2 * GIB, ldh=9000), INVALID), (dict(num_cus=-1), INVALID),
])
def test_plan_norm_rejects(over, status):
    assert status_of(ag.plan_rms_norm, **dict(NORM, **over)) == status


@pytest.mark.parametrize("over", [
    dict(), dict(eps=1e-60), dict(h=A), dict(h=A + 2 * GIB), dict(h=A + 2 * GIB, ldh=9000, ldr=9000), dict(q=None, scale=None), dict(y=None),
    dict(weight=None, residual=None, h=None), dict(y=None, q=None, scale=None, h=None), dict(M=0, x=None, y=None),
    dict(K=0, x=None, q=None), dict(M=1, ldx=1 << 40), dict(x=A + 2, ldx=8193, q=A + 5 * GIB + 1, ldq=8193),
])
def test_plan_norm_accepts(over):
    assert status_of(ag.plan_rms_norm, **dict(NORM, **over)) == ag.AG_OK


@pytest.mark.parametrize("over,status", [
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(rstd=None), INVALID), (dict(rstd=A + 2 * GIB + 2), INVALID),
    (dict(dw_dtype="bf16"), INVALID), (dict(dw_dtype="f32", dw=A + 6 * GIB + 2), INVALID), (dict(accumulate=2), INVALID),
    (dict(dtype="f32"), UNSUPPORTED), (dict(lddx=1), INVALID), (dict(lddh=8191), INVALID), (dict(dx=A), INVALID),
    (dict(dx=A + GIB), INVALID), (dict(dx=A + 4 * GIB + 2), INVALID), (dict(dx=A + 4 * GIB, lddx=9000), INVALID),
    (dict(dw=A + 5 * GIB), INVALID), (dict(dw=A + 4 * GIB), INVALID), (dict(dw=A + 3 * GIB), INVALID), (dict(M=-1), INVALID),
    (dict(M=1 << 31), UNSUPPORTED), (dict(K=(1 << 20) + 1), UNSUPPORTED),
])
def test_plan_norm_backward_rejects(over, status):
    assert status_of(ag.plan_rms_norm_backward, **dict(BACKWARD, **over)) == status


@pytest.mark.parametrize("over", [
    dict(), dict(dh=None), dict(weight=None), dict(dx=None), dict(dw=None), dict(dx=A + 4 * GIB), dict(dw_dtype="f32"),
    dict(accumulate=True), dict(dx=None, dw=None, dy=None, h=None, rstd=None), dict(M=0, dy=None, h=None, rstd=None),
    dict(K=0, dy=None, h=None, rstd=None, dx=None),
])
def test_plan_norm_backward_accepts(over):
    assert status_of(ag.plan_rms_norm_backward, **dict(BACKWARD, **over)) == ag.AG_OK


@pytest.mark.parametrize("over,status", [
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(x=A + 1), INVALID),
    (dict(scale=A + 2 * GIB + 1), INVALID), (dict(M=-1), INVALID), (dict(K=-5), INVALID), (dict(M=1 << 31), UNSUPPORTED),
    (dict(K=(1 << 20) + 1), UNSUPPORTED), (dict(ldx=4095), INVALID), (dict(ldq=4095), INVALID), (dict(ldx=(1 << 20) + 1), UNSUPPORTED),
    (dict(dtype=5), INVALID), (dict(q=A + 100), INVALID), (dict(scale=A), INVALID), (dict(scale=A + GIB), INVALID),
])
def test_quantize_rejects(over, status):
    assert status_of(ag.quantize_rows, **dict(ROWS, **over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(y=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(y=A + 2 * GIB + 2), INVALID),
    (dict(y=A + 8), INVALID), (dict(y=A + GIB), INVALID), (dict(ldy=1), INVALID), (dict(ldq=1), INVALID), (dict(dtype=-1), INVALID),
])
def test_dequantize_rejects(over, status):
    assert status_of(ag.dequantize_rows, **dict(VALUES, **over)) == status


def test_nothing_to_do_needs_no_device():
    ag.quantize_rows(None, None, None, 0, 64, "bf16")
    ag.dequantize_rows(None, None, None, 0, 64, "bf16")
    ag.dequantize_rows(None, A, None, 5, 0, "bf16")
    ag.rms_norm(None, 0, 64, "bf16")
    ag.rms_norm_backward(None, None, None, 0, 64, "bf16")
    ag.rms_norm_backward(A, A + GIB, A + 2 * GIB, 8, 64, "bf16")           # neither gradient is asked for
    ag.rms_norm_backward(None, None, None, 0, 64, "bf16", dw=A, accumulate=True)


def test_reserved_fields_and_null_arguments():
    lib = ag.lib()
    p = ag.RowsPlan()
    assert lib.ag_rms_norm(None, None) == INVALID and lib.ag_rms_norm_backward(None, None, 0, None) == INVALID
    for cls, fn in ((ag.RmsNormArgs, lib.ag_plan_rms_norm), (ag.RmsNormBackwardArgs, lib.ag_plan_rms_norm_backward)):
        a = cls(dtype=ag.AG_BF16)
        if cls is ag.RmsNormArgs:
            a.eps = 1e-6
        else:
            a.dw_dtype = ag.AG_F32
        assert fn(ctypes.byref(a), 256, ctypes.byref(p)) == ag.AG_OK
        assert fn(None, 256, ctypes.byref(p)) == INVALID and fn(ctypes.byref(a), 256, None) == INVALID
        a.reserved[1] = 3
        assert fn(ctypes.byref(a), 256, ctypes.byref(p)) == INVALID


@pytest.mark.parametrize("name,fn,args", [
    ("x", ag.quantize_rows, ROWS), ("q", ag.quantize_rows, ROWS), ("scale", ag.quantize_rows, ROWS), ("y", ag.dequantize_rows, VALUES),
    ("x", ag.plan_rms_norm, NORM), ("weight", ag.plan_rms_norm, NORM), ("q", ag.plan_rms_norm, NORM), ("rstd", ag.plan_rms_norm, NORM),
    ("dy", ag.plan_rms_norm_backward, BACKWARD), ("dw", ag.plan_rms_norm_backward, BACKWARD),
])
def test_tensors_are_checked(name, fn, args):
    """A tensor of another type, or in host memory, is named before its address reaches the library."""
    with pytest.raises(ValueError, match=name):
        fn(**dict(args, **{name: torch.zeros(4, dtype=torch.int32)}))
    right = {"q": torch.int8, "scale": torch.float32, "rstd": torch.float32}.get(name)
    if right is None:
        right = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[args["dtype"]]
    with pytest.raises(ValueError, match=f"{name} does not lie"):
        fn(**dict(args, **{name: torch.zeros(4, dtype=right)}))


def test_workspaces_are_checked():
    with pytest.raises(ValueError, match="workspace"):
        ag.rms_norm_backward(**{k: v for k, v in BACKWARD.items() if k != "num_cus"}, workspace=torch.zeros(1 << 20, dtype=torch.uint8))


def test_plans():
    p = ag.plan_rms_norm(**NORM)
    assert (p.threads_per_row * p.vectors_per_thread * 8 >= 8192 and p.launches == 1 and p.workspace_bytes == 0 and
            1 <= p.n_programs <= 1000)
    assert p.bytes_read == 2 * 2 * 1000 * 8192 + 2 * 8192 and p.bytes_written == 1000 * 8192 * 5 + 8 * 1000
    b = ag.plan_rms_norm_backward(**dict(BACKWARD, dw_dtype="f32"))
    assert b.launches == 2 and b.workspace_bytes >= b.n_programs * 8192 * 4 and b.n_programs <= 1000
    assert b.bytes_read == 3 * 2 * 1000 * 8192 + 4 * 1000 + 2 * 8192 and b.bytes_written == 2 * 1000 * 8192 + 4 * 8192
    assert ag.plan_rms_norm_backward(**dict(BACKWARD, dw=None)).workspace_bytes == 0
    # every row length has threads and registers for all of it, or is read twice
    for K in [1, 128, 129, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385, 32768, 32769, 1 << 20]:
        p = ag.plan_rms_norm(**dict(NORM, K=K, M=3))
        assert p.vectors_per_thread == 0 or p.threads_per_row * p.vectors_per_thread * 8 >= K


# ------------------------------------------------------------------ the oracle

def nearest_even(f: Fraction) -> int:
    return round(f)         # of a Fraction: to nearest, ties to even


def test_quantize_oracle_is_exact():
    g = np.random.default_rng(1)
    for scale in (1.0, 2.0 ** -30, 2.0 ** 40):
        v = torch.from_numpy(g.standard_normal((4, 60)) * scale).to(torch.float32).double().numpy()
        codes, scales = quantize_oracle(v)
        for row, c, s in zip(v, codes, scales):
            top = max(abs(Fraction(float(t))) for t in row)
            assert [nearest_even(Fraction(float(t)) * 127 / top) for t in row] == c.tolist()
            assert abs(Fraction(float(s)) * 127 - top) <= top * Fraction(1, 2 ** 52)


def test_quantize_oracle_ties_zeros_and_what_is_not_finite():
    codes, scales = quantize_oracle(np.array([[254.0, 1.0, 3.0, -1.0, -5.0], [0.0] * 5, [1.0, np.nan, 2.0, 0.0, 0.0],
                                              [np.inf, 1.0, 0.0, 0.0, 0.0]]))
    assert codes.tolist() == [[127, 0, 2, 0, -2], [0] * 5, [0] * 5, [0] * 5]
    assert scales[0] == 2.0 and scales[1] == 0.0 and np.isnan(scales[2:]).all()


def test_norm_oracle():
    h = np.array([[3.0, 4.0], [0.0, 0.0]])
    y, rstd, codes, scales = norm_oracle(h, np.array([2.0, 1.0]), 0.5)
    assert np.allclose(rstd, [1 / np.sqrt(13.0), 1 / np.sqrt(0.5)]) and np.allclose(y[0], [6 / np.sqrt(13), 4 / np.sqrt(13)])
    assert codes.tolist() == [[127, 85], [0, 0]] and np.allclose(scales, [6 / 127 / np.sqrt(13), 0.0])
    # autograd of the same formula
    g = np.random.default_rng(2)
    h, w, dy, dh = (torch.from_numpy(g.standard_normal(s)) for s in ((5, 33), (33,), (5, 33), (5, 33)))
    h.requires_grad_(), w.requires_grad_()
    r = (h.square().mean(1) + 1e-3).rsqrt()
    (h * r[:, None] * w * dy + h * dh).sum().backward()
    dx, dw = norm_backward_oracle(dy.numpy(), h.detach().numpy(), r.detach().numpy(), w.detach().numpy(), dh.numpy())
    assert np.allclose(dx, h.grad.numpy(), rtol=1e-12) and np.allclose(dw, w.grad.numpy(), rtol=1e-12)


def test_codes_product_oracle():
    x, w = np.array([[1, -2], [127, 127]], dtype=np.int8), np.array([[3, 4], [-128, 127]], dtype=np.int8)
    got = codes_product_oracle(x, w, np.array([1.0, 0.5], np.float32), np.array([2.0, 1.0], np.float32))
    assert got.tolist() == [[-10.0, -382.0], [889.0, -63.5]]


# ------------------------------------------------------------------ generated code

def test_row_kernels_never_spill(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "gemm_all_gather_amd", "csrc")

    def kernels(name):
        out = str(tmp_path / (name + ".s"))
        subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", f"-I{csrc}", f"-I{os.path.join(root, 'include')}", "--cuda-device-only",
                        "-S", "-o", out, os.path.join(csrc, name + ".hip")], check=True, capture_output=True)
        return re.findall(r"\.amdhsa_kernel (\S+)\n.*?private_segment_fixed_size (\d+)", open(out).read(), re.S)

    with ThreadPoolExecutor(3) as pool:
        found = sum(pool.map(kernels, ("ag_rows", "ag_linear_i8", "ag_linear_q8")), [])
    assert len(found) > 100 and all(int(scratch) == 0 for _, scratch in found), [f for f in found if int(f[1])]
