"""What the plans of the 8-bit operators say about the kernels that run, without a GPU."""

import pytest

from gemm_all_gather_amd import binding as ag
from tests.test_linear_cpu import A, GIB

FORWARD = dict(x=A, w=A + GIB, x_scale=A + 6 * GIB, w_scale=A + 7 * GIB, y=A + 2 * GIB, N=1024, K=4096, dtype="bf16", num_cus=256)


@pytest.mark.parametrize("M,rows,width", [(1, 16, 256), (16, 16, 256), (17, 32, 128), (32, 32, 128), (33, 64, 64), (48, 64, 64), (64, 64, 64)])
def test_streamed_shape(M, rows, width):
    """16, 32 or 64 rows of x to a workgroup, and the more of them, the shorter a wave's part of the reduction."""
    p = ag.plan_linear_i8(M=M, **FORWARD).product
    assert (p.variant, p.tile_m, p.tile_n, p.tile_k) == (1, rows, 16, width)
    assert p.n_programs == 1024 // 16
