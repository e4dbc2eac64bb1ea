"""What the linear layer's plans say of workspaces and launches, without a GPU."""

from gemm_all_gather_amd import binding as ag
from tests.test_linear_cpu import BACKWARD


def test_an_fp32_weight_gradient_behind_an_activation_takes_dz_in_two_terms():
    M, N = BACKWARD["M"], BACKWARD["N"]
    dz = (2 * M * N + 255) // 256 * 256
    for act in ("gelu", "gelu_tanh", "silu"):
        alone = dict(BACKWARD, act=act, dx=None, db=None, w=None)
        one, two = (ag.plan_linear_backward(**dict(alone, dw_dtype=t)) for t in ("f16", "f32"))
        assert two.workspace_bytes == one.workspace_bytes + dz
        assert two.launches - 1 == 2 * (one.launches - 1)       # the slope's launch, then every product's
        assert two.flops == one.flops
    # one term where nothing is rounded, or where fp32 is not asked for
    for over in (dict(act="none", z=None), dict(act="relu")):
        one, same = (ag.plan_linear_backward(**dict(BACKWARD, dw_dtype=t, **over)) for t in ("f16", "f32"))
        assert (one.workspace_bytes, one.launches) == (same.workspace_bytes, same.launches)
    none, same = (ag.plan_linear_backward(**dict(BACKWARD, dw=None, x=None, dw_dtype=t)) for t in ("f16", "f32"))
    assert (none.workspace_bytes, none.launches) == (same.workspace_bytes, same.launches)
