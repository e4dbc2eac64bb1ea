"""The fp16 product kernels' generated code: every fragment read is waited for on every path, and nothing spills.

(The bf16 ones' is checked beside the plans; the two are compiled apart, and a register may be chosen otherwise.)
"""

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_linear_cpu import unwaited_uses


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "gemm_all_gather_amd", "csrc")
    tmp = tmp_path_factory.mktemp("isa_f16")

    def compile_one(name):
        out = str(tmp / (name + ".s"))
        subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", f"-I{csrc}", f"-I{os.path.join(root, 'include')}", "--cuda-device-only",
                        "-S", "-o", out, os.path.join(csrc, name + ".hip")], check=True, capture_output=True)
        return open(out).read()

    with ThreadPoolExecutor(2) as pool:
        return "\n".join(pool.map(compile_one, ("ag_linear_forward_f16", "ag_linear_grads_f16")))


def test_fp16_product_kernels_wait_for_fragments_and_never_spill(asm):
    kernels = re.findall(r"^(_Z\S*ag_linear_(?:gemm|grads)\S*):", asm, re.M)
    assert len(kernels) == 15 + 6 + 3     # 5 activations, 2 gradients in 3 tiles; in turn either way, side by side
    for k in kernels:
        start = asm.index(f"\n{k}:")
        lines = [ln.split(";", 1)[0].strip() for ln in asm[start:asm.index(".section", start)].splitlines()]
        lines = [ln for ln in lines if ln]
        assert sum(ln.startswith("v_mfma") for ln in lines) >= 32, k
        assert sum(ln.startswith("ds_read") for ln in lines) >= 16, k
        assert not unwaited_uses(lines), (k, unwaited_uses(lines)[:3])
        meta = re.search(r"\.amdhsa_kernel " + re.escape(k) + r"\n(.*?)\.end_amdhsa_kernel", asm, re.S).group(1)
        assert re.search(r"private_segment_fixed_size 0\n", meta), k
