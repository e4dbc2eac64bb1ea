"""What the linear layer's plans say of workspaces and launches, without a GPU."""

from gemm_all_gather_amd import binding as ag
from tests.test_linear_cpu import BACKWARD, FORWARD
from tests.test_linear_reach_gpu import FEW_ROWS, IN_TURN, ROUNDS, TILES


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


def rounds_up(a, b):
    return -(-a // b)


def test_the_reach_tests_sizes_reach_what_they_are_for():
    """On 256 CUs: the streaming kernel's forms and rounds, tiles whole and cut, uneven deals of gradients in turn."""
    seen = set()
    for M, N, K in FEW_ROWS:
        p = ag.plan_linear(**dict(FORWARD, M=M, N=N, K=K)).product
        assert p.variant == 1
        waves = 16 if p.n_programs <= 256 else 8
        blocks = rounds_up(K // 128, waves)         # of the first wave
        assert blocks >= 2, (M, N, K)               # a second block is on its way while the first is multiplied
        seen.add((waves, M > 16, "more" if blocks > 2 else "two", "tail" if K % 128 else "whole"))
    for waves in (16, 8):
        for form in (False, True):
            assert any(s[:2] == (waves, form) for s in seen), (waves, form)
        assert any(s[0] == waves and s[2] == "more" for s in seen) and any(s[0] == waves and s[3] == "tail" for s in seen)
    assert any(s[3] == "whole" for s in seen)
    for tile, (M, N, K) in TILES.items():
        p = ag.plan_linear(**dict(FORWARD, M=M, N=N, K=K)).product
        assert (p.tile_m, p.tile_n) == tile and p.splits == 1
    kinds = set()
    for M, N, K, dtype, _ in ROUNDS:
        p = ag.plan_linear(**dict(FORWARD, M=M, N=N, K=K)).product
        kinds.add((p.tile_m, p.tile_n, p.splits > 1, dtype))
        assert p.full_tiles >= 256
        if p.splits == 1:
            assert p.full_tiles > 3 * 256
    assert kinds >= {(256, 256, True, "f16"), (256, 256, True, "bf16"), (256, 256, False, "bf16"), (256, 128, True, "f16"),
                     (256, 128, True, "bf16")}
    orders = set()
    for M, N, K in IN_TURN:
        b = ag.plan_linear_backward(**dict(BACKWARD, M=M, N=N, K=K, act="none", z=None, dw_dtype="f32"))
        assert b.launches == 2 and b.product.tile_m == b.product_dw.tile_m == 256       # after db's column sums
        dx_first = N >= M
        first, second = (b.product, b.product_dw) if dx_first else (b.product_dw, b.product)
        heavy = first.full_tiles % 256
        # left to the workgroups without a tile of the first, the second's tiles take longer than a round on all of them
        # after the first's longer tile, the rest again on those without
        long, short = (rounds_up(r, 64) for r in ((N, M) if dx_first else (M, N)))
        light = 256 - heavy
        apart = rounds_up(second.full_tiles, light) * short
        shared = max(long + short, (1 + rounds_up(second.full_tiles - 256, light)) * short)
        assert heavy and second.full_tiles > 256 and shared < apart, (M, N, K)
        orders.add(dx_first)
    assert orders == {True, False}
