"""The linear layer's gradients from activations kept in 8 bits without a GPU: refusals and plans."""

import ctypes

import pytest
import torch

from gemm_all_gather_amd import binding as ag
from tests.test_linear_cpu import A, GIB, INVALID, UNSUPPORTED, status_of

BACKWARD = dict(dy=A, x=A + GIB, w=A + 2 * GIB, z=A + 3 * GIB, dx=A + 4 * GIB, dw=A + 5 * GIB, db=A + 6 * GIB, x_scale=A + 7 * GIB,
                z_scale=A + 8 * GIB, M=1000, N=3584, K=8192, dtype="f16", act="silu", num_cus=256)


@pytest.mark.parametrize("over,status", [
    (dict(dy=None), INVALID), (dict(z=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(x_scale=A + 7 * GIB + 2), INVALID), (dict(z_scale=A + 8 * GIB + 1), INVALID), (dict(dw_dtype="bf16"), INVALID),
    (dict(ldx=8191), INVALID), (dict(ldz=3583), INVALID), (dict(dtype="f32"), UNSUPPORTED), (dict(dx=A + GIB), INVALID),
    (dict(dw=A + 7 * GIB), INVALID), (dict(dx=A + 8 * GIB - 100), INVALID), (dict(db=A + 8 * GIB + 16), INVALID),
    (dict(x=A + 4 * GIB + 1000 * 8192 * 2 - 1), INVALID), (dict(accumulate=2), INVALID), (dict(act=9), INVALID),
])
def test_rejects(over, status):
    assert status_of(ag.plan_linear_backward_q8, **dict(BACKWARD, **over)) == status


@pytest.mark.parametrize("over", [
    dict(), dict(x_scale=None), dict(z_scale=None), dict(x_scale=None, z_scale=None), dict(x=A + GIB + 1, ldx=8193),
    dict(act="none", z=None, z_scale=None), dict(act="none", z=None), dict(dw=None, x=None), dict(dw=None, x=None, x_scale=None),
    dict(dx=None, w=None), dict(M=0, dy=None, z=None, x=None), dict(dx=None, dw=None, db=None, dy=None, x=None, w=None, z=None),
    # codes of one byte end before what 16 bits would reach
    dict(x=A + 4 * GIB + 1000 * 8192 * 2), dict(x=A + 4 * GIB - 1000 * 8192),
])
def test_accepts(over):
    assert status_of(ag.plan_linear_backward_q8, **dict(BACKWARD, **over)) == ag.AG_OK


def test_null_arguments():
    lib, p = ag.lib(), ag.LinearPlan()
    assert lib.ag_linear_backward_q8(None, None, None, None, 0, None) == INVALID
    assert lib.ag_plan_linear_backward_q8(None, None, None, 256, ctypes.byref(p)) == INVALID
    a = ag.LinearBackwardArgs(dtype=ag.AG_BF16, dw_dtype=ag.AG_F32)
    assert lib.ag_plan_linear_backward_q8(ctypes.byref(a), None, None, 256, None) == INVALID
    a.reserved[2] = 1
    assert lib.ag_plan_linear_backward_q8(ctypes.byref(a), None, None, 256, ctypes.byref(p)) == INVALID


@pytest.mark.parametrize("name", ["dy", "x", "w", "z", "dx", "dw", "db", "x_scale", "z_scale"])
def test_tensors_are_checked(name):
    with pytest.raises(ValueError, match=name):
        ag.plan_linear_backward_q8(**dict(BACKWARD, **{name: torch.zeros(4, dtype=torch.int32)}))
    right = torch.int8 if name in ("x", "z") else torch.float32 if "scale" in name else torch.float16
    with pytest.raises(ValueError, match=f"{name} does not lie"):
        ag.plan_linear_backward_q8(**dict(BACKWARD, **{name: torch.zeros(4, dtype=right)}))


def test_plans():
    fields = lambda p: [(n, bytes(getattr(p, n)) if "product" in n else getattr(p, n)) for n, _ in p._fields_]  # noqa: E731
    none = dict(BACKWARD, x_scale=None, z_scale=None)
    same = ag.plan_linear_backward_q8(**none)
    plain = ag.plan_linear_backward(**{k: v for k, v in none.items() if "scale" not in k})
    assert fields(same) == fields(plain)
    both = ag.plan_linear_backward_q8(**BACKWARD)
    M, N, K = 1000, 3584, 8192
    assert both.bytes_read == 2 * M * N + M * N + 4 * M + M * K + 4 * M + 2 * N * K and both.flops == 4.0 * M * N * K
    assert both.bytes_written == plain.bytes_written and both.launches == plain.launches
    # dz for dx, dz with the scale's factor for dw, x's codes in 16 bits
    assert both.workspace_bytes >= 2 * (2 * M * N + M * K)
    z_only = ag.plan_linear_backward_q8(**dict(BACKWARD, x_scale=None))
    assert z_only.workspace_bytes == plain.workspace_bytes and z_only.launches == plain.launches


@pytest.mark.parametrize("dtype,terms", [("f16", 2), ("bf16", 3)])
@pytest.mark.parametrize("M", [1, 200, 32 * 200 + 31, 32 * 200 + 32])
def test_terms_of_a_wide_weight_gradient(M, dtype, terms):
    """dw in fp32: dz's terms in one product with as many copies of x, or, of few columns, a product each."""
    N, K = 200, 256         # rows of dz's terms take 256 elements, those of x's values 256
    wide = ag.plan_linear_backward_q8(**dict(BACKWARD, M=M, N=N, K=K, dtype=dtype, dw_dtype="f32", dx=None, w=None, db=None))
    dz, x = 2 * M * 256 * terms, 2 * M * K
    if M // 32 <= N:
        assert wide.workspace_bytes >= dz + terms * x and wide.launches <= 3        # codes and terms, the product, its join
    else:
        assert wide.launches >= 1 + terms       # (cut tiles' sums are in the workspace too, so its size says nothing here)
