"""The linear layer on 8-bit integers with scales at fp32's ends, against exact sums: no intermediate leaves fp32's range
where the result is inside it, whatever the order of sum, row scale and column scale."""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from tests.gpu_util import log, require_gpu
from tests.test_linear_i8_gpu import Layer

pytestmark = pytest.mark.gpu

# streamed; in tiles, whole and ragged ones; with cut reductions and their join
SHAPES = [(3, 70, 64), (90, 70, 64), (128, 128, 192), (300, 264, 2200)]
# (row, column): sums here are up to 2^22
SCALES = [(2.0 ** 115, 2.0 ** -115), (2.0 ** -115, 2.0 ** 115), (2.0 ** -100, 2.0 ** -40), (2.0 ** -40, 2.0 ** -100), (1.5 * 2.0 ** 95, 2.0 ** 3),
          (2.0 ** 127, 2.0 ** -127), (1.5 * 2.0 ** 127, 3 * 2.0 ** -149), (1.5 * 2.0 ** -140, 2.0 ** 120), (2.0 ** -149, 2.0 ** 127),
          (2.0 ** -127, 2.0 ** 125), (-(2.0 ** 115), 2.0 ** -115), (2.0 ** 60, 2.0 ** -60), (1.0, 1.0)]


def test_a_shape_has_cut_reductions():
    require_gpu()
    f = Layer(*SHAPES[-1], "bf16", residual=False, z=False)
    assert ag.plan_linear_i8(**f.args()).product.splits > 1


@pytest.mark.parametrize("row,column", SCALES)
def test_products_of_scales(row, column):
    require_gpu()
    for M, N, K in SHAPES:
        for z in (False, True):
            what = f"linear_i8 {M}x{N}x{K} row scales {row} column scales {column} z {z}"
            log(what)
            f = Layer(M, N, K, "bf16", bias=False, residual=False, z=z)
            f.xs.view.fill_(row)
            f.ws.view.fill_(column)
            f.run()
            f.check(what)


def test_sums_of_zero_stay_zero():
    """Whatever finite scales stand beside them."""
    require_gpu()
    for M, N, K in SHAPES:
        for row, column in ((1.9 * 2.0 ** 127, 1.9 * 2.0 ** 127), (2.0 ** -149, 2.0 ** -149)):
            log(f"linear_i8 {M}x{N}x{K} of zeros, scales {row} and {column}")
            f = Layer(M, N, K, "bf16", bias=False, residual=False, z=False)
            f.x.view.zero_()
            f.xs.view.fill_(row)
            f.ws.view.fill_(column)
            f.run()
            torch.cuda.synchronize()
            assert not f.y.f64().any()


def test_rows_of_every_size():
    """Each row its own scale from 2^-149 to 2^127, beside columns that bring the result back, all in one call."""
    require_gpu()
    for M, N, K in SHAPES:
        log(f"linear_i8 {M}x{N}x{K} with rows of every size")
        f = Layer(M, N, K, "bf16", bias=False, residual=False, z=False)
        f.xs.view.copy_(torch.from_numpy(np.exp2(np.linspace(-149, 80, M).round())[None]).float())
        f.ws.view.fill_(2.0 ** 20)
        f.run()
        f.check("rows of every size")


def test_results_past_fp32_are_infinite():
    require_gpu()
    for M, N, K in SHAPES[:2]:
        log(f"linear_i8 {M}x{N}x{K} past fp32's largest")
        f = Layer(M, N, K, "bf16", bias=False, residual=False, z=False)
        f.x.view.fill_(1), f.w.view.fill_(1)
        f.w.view[1] = -1
        f.xs.view.fill_(2.0 ** 100)
        f.ws.view.fill_(2.0 ** 60)
        f.run()
        torch.cuda.synchronize()
        y = f.y.f64()
        assert np.isneginf(y[:, 1]).all() and np.isposinf(np.delete(y, 1, 1)).all()
