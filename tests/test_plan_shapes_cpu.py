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


BACKWARD = dict(dy=A, x=A + 100 * GIB, w=A + 200 * GIB, dx=A + 400 * GIB, dw=A + 500 * GIB, x_scale=A + 700 * GIB, num_cus=256, dw_dtype="f32")


@pytest.mark.parametrize("dtype,terms", [("f16", 2), ("bf16", 3)])
@pytest.mark.parametrize("M,N,K", [(2048, 3584, 8192), (4096, 3584, 8192), (4097, 3584, 8192), (8192, 3584, 8192), (16384, 3584, 8192),
                                   (16384, 1024, 4096), (65536, 4096, 4096)])
def test_copies_of_kept_rows_are_bounded(M, N, K, dtype, terms):
    """x's values for dw in fp32: a copy per term only while those past the first take at most 128 MiB."""
    a = dict(BACKWARD, M=M, N=N, K=K, dtype=dtype)
    apart = ag.plan_linear_backward_q8(**dict(a, dw_dtype=dtype))       # one term, one copy
    wide = ag.plan_linear_backward_q8(**a)
    copy, term = 2 * M * K, 2 * M * N
    partial = 512 << 20         # cut tiles' sums are bounded by themselves
    assert wide.workspace_bytes <= terms * term + copy + (128 << 20) + partial
    if (terms - 1) * copy > 128 << 20:
        assert wide.launches >= apart.launches + terms - 1
        assert wide.workspace_bytes <= apart.workspace_bytes + (terms - 1) * term + partial
    else:
        assert wide.workspace_bytes >= terms * (term + copy)


@pytest.mark.parametrize("M,N", [(159, 4), (160, 4), (6431, 200), (6432, 200)])
def test_narrow_weight_gradients_take_a_product_a_term(M, N):
    """From M = 32 (N + 1) on."""
    wide = ag.plan_linear_backward_q8(**dict(BACKWARD, M=M, N=N, K=256, dtype="bf16", dx=None, w=None))
    assert (wide.launches >= 4) == (M >= 32 * (N + 1))
