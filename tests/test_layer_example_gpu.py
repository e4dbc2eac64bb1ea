"""The layer training example: all-gather, linear, linear_backward and AdamW together on the logical ranks."""

import pytest
import torch

from examples.layer_training_step import train
from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu


def test_the_example_layer_learns_and_serves():
    require_gpu()
    log("layer training example")
    losses, out, want = train(steps=25, world=4, rows=64, features=256, outputs=520)
    assert len(losses) == 25 and losses[-1] < 0.25 * losses[0], losses
    # the token's and the batch's kernels sum in different orders: one rounding to bf16 apart at most
    assert torch.all((out - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12)
    again, _, _ = train(steps=3, world=4, rows=64, features=256, outputs=520)
    assert again == losses[:3]                  # the same run twice: the same bits
