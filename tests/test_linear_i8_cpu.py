"""The linear layer on 8-bit integers without a GPU: refusals, plans, and its kernels' generated code."""

import ctypes
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from gemm_all_gather_amd import binding as ag
from tests.linear_util import HUGE, LARGE
from tests.test_linear_cpu import A, GIB, INVALID, UNSUPPORTED, status_of, unwaited_uses

FORWARD = dict(x=A, w=A + GIB, x_scale=A + 6 * GIB, w_scale=A + 7 * GIB, y=A + 2 * GIB, M=1000, N=3584, K=8192, dtype="bf16", act="gelu",
               bias=A + 3 * GIB, residual=A + 4 * GIB, z=A + 5 * GIB, num_cus=256)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(x_scale=None), INVALID), (dict(w_scale=None), INVALID),
    (dict(x_scale=A + 6 * GIB + 2), INVALID), (dict(w_scale=A + 7 * GIB + 1), INVALID), (dict(bias=A + 3 * GIB + 1), INVALID),
    (dict(y=A + 2 * GIB + 1), INVALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(dtype="f32"), UNSUPPORTED), (dict(dtype=7), INVALID), (dict(act=5), INVALID),
    (dict(ldx=8191), INVALID), (dict(ldw=100), INVALID), (dict(ldy=3583), INVALID), (dict(ldr=1), INVALID), (dict(ldz=-3584), INVALID),
    (dict(M=1 << 31), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=131072), UNSUPPORTED), (dict(ldx=(1 << 20) + 1), UNSUPPORTED),
    (dict(y=A + 1000), INVALID), (dict(y=A + GIB), INVALID), (dict(z=A + 2 * GIB), INVALID), (dict(z=A + 4 * GIB), INVALID),
    (dict(y=A + 6 * GIB), INVALID), (dict(z=A + 7 * GIB + 4), INVALID), (dict(y=A + 4 * GIB + 2), INVALID),
    (dict(y=A + 4 * GIB, ldy=3600), INVALID), (dict(num_cus=-1), INVALID),
])
def test_plan_linear_i8_rejects(over, status):
    assert status_of(ag.plan_linear_i8, **dict(FORWARD, **over)) == status


@pytest.mark.parametrize("over", [
    dict(), dict(bias=None, residual=None, z=None), dict(y=A + 4 * GIB), dict(x=A + 1, w=A + GIB + 3), dict(ldx=9001),
    dict(M=0, x=None, y=None, x_scale=None), dict(N=0, w=None, y=None, w_scale=None), dict(K=0, x=None, w=None), dict(M=1, ldx=1 << 40),
    dict(K=131071), dict(M=100, N=1 << 20, K=16),
])
def test_plan_linear_i8_accepts(over):
    assert status_of(ag.plan_linear_i8, **dict(FORWARD, **over)) == ag.AG_OK


def test_reserved_fields_and_null_arguments():
    lib, p = ag.lib(), ag.LinearPlan()
    assert lib.ag_linear_i8(None, None, 0, None) == INVALID and lib.ag_plan_linear_i8(None, 256, ctypes.byref(p)) == INVALID
    a = ag.LinearI8Args(dtype=ag.AG_BF16)
    assert lib.ag_plan_linear_i8(ctypes.byref(a), 256, None) == INVALID
    assert lib.ag_plan_linear_i8(ctypes.byref(a), 256, ctypes.byref(p)) == ag.AG_OK and p.launches == 0
    a.reserved[5] = 1
    assert lib.ag_plan_linear_i8(ctypes.byref(a), 256, ctypes.byref(p)) == INVALID


@pytest.mark.parametrize("name", ["x", "w", "x_scale", "w_scale", "bias", "residual", "y", "z"])
def test_tensors_are_checked(name):
    with pytest.raises(ValueError, match=name):
        ag.plan_linear_i8(**dict(FORWARD, **{name: torch.zeros(4, dtype=torch.int32)}))
    right = torch.int8 if name in "xw" else torch.float32 if "scale" in name else torch.bfloat16
    with pytest.raises(ValueError, match=f"{name} does not lie"):
        ag.plan_linear_i8(**dict(FORWARD, **{name: torch.zeros(4, dtype=right)}))


def test_plans():
    p = ag.plan_linear_i8(**FORWARD)
    assert p.flops == 2.0 * 1000 * 3584 * 8192 and p.product.variant == 2 and p.product.tile_k == 128 and p.product.packed == 0
    assert p.bytes_read == 1000 * 8192 + 3584 * 8192 + 4 * 4584 + 2 * (3584 + 1000 * 3584) and p.bytes_written == 4 * 1000 * 3584
    one = ag.plan_linear_i8(**dict(FORWARD, M=1))
    assert one.product.variant == 1 and one.workspace_bytes == 0 and one.launches == 1
    # copies of rows that do not start on 4 bytes
    odd = ag.plan_linear_i8(**dict(FORWARD, K=8191))
    assert odd.product.packed == 3 and odd.launches >= 2 and odd.workspace_bytes >= (1000 + 3584) * 8192
    assert ag.plan_linear_i8(**dict(FORWARD, x=A + 2)).product.packed == 1
    assert ag.plan_linear_i8(**dict(FORWARD, ldw=8194)).product.packed == 2
    assert ag.plan_linear_i8(**dict(FORWARD, x=A + 4, ldw=8196)).product.packed == 0


def test_sizes_reach_every_tile_whole_and_cut():
    """The sizes of the GPU tests run every tile kind, with and without cut reductions."""
    seen = set()
    for M, N, K in LARGE + HUGE + [(700, 700, 20000), (300, 264, 16001), (128, 128, 192), (257, 300, 520)]:
        p = ag.plan_linear_i8(A, A + 64 * GIB, A + 128 * GIB, A + 129 * GIB, A + 130 * GIB, M, N, K, "bf16", num_cus=256).product
        if p.variant == 2:
            seen.add((p.tile_m, p.tile_n, p.splits > 1))
            assert 1 <= p.n_programs <= 256 and (p.splits == 1) == (p.full_tiles == -(-M // p.tile_m) * -(-N // p.tile_n))
    log = sorted(seen)
    assert {(m, n) for m, n, _ in seen} == {(256, 256), (256, 128), (128, 128)} and any(s for _, _, s in seen), log


# ------------------------------------------------------------------ generated code

@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "gemm_all_gather_amd", "csrc")
    tmp = tmp_path_factory.mktemp("isa_i8")

    def compile_one(name):
        out = str(tmp / (name + ".s"))
        subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", f"-I{csrc}", f"-I{os.path.join(root, 'include')}", "--cuda-device-only",
                        "-S", "-o", out, os.path.join(csrc, name + ".hip")], check=True, capture_output=True)
        return open(out).read()

    with ThreadPoolExecutor(2) as pool:
        return "\n".join(pool.map(compile_one, ("ag_linear_i8_f16", "ag_linear_i8_bf16")))


def test_kernels_wait_for_fragments_and_never_spill(asm):
    kernels = re.findall(r"^(_Z\S*ag_linear_i8_gemm\S*):", asm, re.M)
    assert len(kernels) == 2 * 5 * 3      # types, activations, tiles
    for k in kernels:
        start = asm.index(f"\n{k}:")
        lines = [ln.split(";", 1)[0].strip() for ln in asm[start:asm.index(".section", start)].splitlines()]
        lines = [ln for ln in lines if ln]
        assert sum(ln.startswith("v_mfma_i32_16x16x64_i8") for ln in lines) >= 32, k
        assert sum(ln.startswith("ds_read") for ln in lines) >= 16, k
        assert not unwaited_uses(lines), (k, unwaited_uses(lines)[:3])
        meta = re.search(r"\.amdhsa_kernel " + re.escape(k) + r"\n(.*?)\.end_amdhsa_kernel", asm, re.S).group(1)
        assert re.search(r"private_segment_fixed_size 0\n", meta), k
