"""The linear layer's kernels that no other size reaches.

Few rows: the streaming kernel's loop round after round, with sixteen and with eight waves a workgroup.  Tiles: every
activation in every tile and type, cut reductions after whole rounds, whole rounds alone; and gradients in turn where the
workgroups with a tile less of the first product take more of the second's.
"""

import pytest

from gemm_all_gather_amd import binding as ag
from tests.gpu_util import log, require_gpu
from tests.test_linear_gpu import ACTS, Backward, Forward

pytestmark = pytest.mark.gpu

# M, N, K.  Sixteen waves (up to 256 workgroups of 16 rows of w) share 2048 of K a round, eight 1024.
FEW_ROWS = [(1, 3584, 8192), (16, 4096, 4104), (16, 520, 6300), (32, 520, 8200), (17, 1000, 4200),
            (1, 4113, 2440), (13, 4112, 3584), (16, 5000, 4099), (20, 4200, 1900), (32, 4100, 1990)]
TILES = {(256, 256): (8300, 1100, 200), (256, 128): (2100, 2300, 520), (128, 128): (700, 500, 264)}
# whole rounds of 256 x 256 tiles, the others cut or not; 256 x 128 tiles cut
ROUNDS = [(4352, 4000, 4096, "f16", "relu"), (4352, 4000, 4096, "bf16", "none"), (6144, 8704, 520, "bf16", "silu"),
          (4352, 2048, 8192, "f16", "none"), (2048, 4352, 8192, "bf16", "relu")]
# dx first, and dw first
IN_TURN = [(830, 1580, 10030), (1790, 1000, 9900)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", FEW_ROWS)
def test_few_rows_round_after_round(M, N, K, dtype):
    require_gpu()
    for pad, offset, act in ((0, 0, "silu"), (3, 1, "none")):
        what = f"linear {M}x{N}x{K} {dtype} {act} pad {pad} offset {offset}"
        log(what)
        f = Forward(M, N, K, dtype, act, pad=pad, offset=offset, seed=5)
        f.run()
        f.check(what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("tile", list(TILES))
def test_every_activation_in_every_tile(tile, act, dtype):
    require_gpu()
    f = Forward(*TILES[tile], dtype, act, seed=6)
    p = ag.plan_linear(**f.args()).product
    what = f"linear {TILES[tile]} {dtype} {act} tile {p.tile_m}x{p.tile_n}"
    log(what)
    f.run()
    f.check(what)


@pytest.mark.parametrize("M,N,K,dtype,act", ROUNDS)
def test_whole_rounds_and_cut_ones(M, N, K, dtype, act):
    require_gpu()
    f = Forward(M, N, K, dtype, act, seed=7)
    p = ag.plan_linear(**f.args()).product
    what = f"linear {M}x{N}x{K} {dtype} {act}: tile {p.tile_m}x{p.tile_n} full {p.full_tiles} splits {p.splits}"
    log(what)
    f.run()
    f.check(what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", IN_TURN)
def test_gradients_in_turn_dealt_unevenly(M, N, K, dtype):
    require_gpu()
    b = Backward(M, N, K, dtype, "none", "f32" if dtype == "bf16" else None, accumulate=True, seed=8)
    what = f"linear_backward {M}x{N}x{K} {dtype}"
    log(what)
    b.run()
    b.check(what)
