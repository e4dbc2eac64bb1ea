"""The linear layer's workspace: nothing beyond the plan's bytes is touched, on any stream, and what is refused.

The workspace's contents before a call must not matter, so it is filled with NaN patterns; the fill and the call are
ordered by events where they are on different streams, and the workspace lives until both have ended.
"""

import pytest
import torch

from gemm_all_gather_amd import binding as ag
from tests.gpu_util import log, require_gpu
from tests.test_linear_gpu import Backward, Forward

pytestmark = pytest.mark.gpu

GUARD = 1 << 16
FORWARD = [(33, 600, 4100), (513, 520, 2048), (700, 700, 8192), (300, 264, 1100)]
BACKWARD = [(33, 600, 4100), (513, 264, 520), (1100, 8300, 600), (150, 264, 200), (1000, 1030, 2050)]


class Workspace:
    """The plan's bytes between two guards."""

    def __init__(self, nbytes):
        self.nbytes = nbytes
        self.all = torch.full((2 * GUARD + nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
        self.all[:GUARD] = self.all[GUARD + nbytes:] = 0x5A

    @property
    def view(self):
        return self.all[GUARD:GUARD + self.nbytes]

    def check(self, what):
        assert bool((self.all[:GUARD] == 0x5A).all()) and bool((self.all[GUARD + self.nbytes:] == 0x5A).all()), \
            f"{what}: written outside the workspace"


def run_twice(side, call, ws, op, what):
    """Two calls on the side stream, each after a fill of the workspace on the current one, give the same bits."""
    first = None
    for _ in range(2):
        ws.view.fill_(0xFF)
        side.wait_stream(torch.cuda.current_stream())
        log(what)
        call()
        torch.cuda.synchronize()
        ws.check(what)
        op.check(what)
        bits = [m.buffer.view(torch.int32 if m.dtype == "f32" else torch.int16).clone() for m in op.outputs]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, bits)), what
        first = bits


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_linear_stays_inside_its_workspace(M, N, K, pad):
    require_gpu()
    f = Forward(M, N, K, "bf16", "gelu", pad=pad, seed=9)
    f.outputs = [f.y, f.z]
    ws = Workspace(ag.plan_linear(**f.args()).workspace_bytes)
    assert ws.nbytes or pad == 0
    side = torch.cuda.Stream()
    run_twice(side, lambda: ag.linear(**f.args(), workspace=ws.view, stream=side), ws, f, f"linear {M}x{N}x{K} pad {pad}")


@pytest.mark.parametrize("dw", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_linear_backward_stays_inside_its_workspace(M, N, K, pad, dw):
    require_gpu()
    b = Backward(M, N, K, "bf16", "silu", dw, pad=pad, seed=9)
    b.outputs = [b.dx, b.dw, b.db]
    ws = Workspace(ag.plan_linear_backward(**b.args()).workspace_bytes)
    assert ws.nbytes
    side = torch.cuda.Stream()
    run_twice(side, lambda: ag.linear_backward(**b.args(), workspace=ws.view, stream=side), ws, b,
              f"linear_backward {M}x{N}x{K} pad {pad} dw {dw}")


def refused(call, **k):
    with pytest.raises(ag.AgError, match="workspace") as exc:
        call(**k)
    assert exc.value.status == ag.AG_ERR_INVALID_ARG


@pytest.mark.parametrize("op", ["linear", "linear_backward"])
def test_workspaces_that_are_refused(op):
    """All found on the host, before a launch."""
    require_gpu()
    o = Forward(300, 264, 1100, "bf16", "gelu") if op == "linear" else Backward(300, 264, 1100, "bf16", "gelu")
    call, plan = (ag.linear, ag.plan_linear) if op == "linear" else (ag.linear_backward, ag.plan_linear_backward)
    args = o.args()
    need = plan(**args).workspace_bytes
    assert need > 0
    ws = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    log(f"{op}: refused workspaces")
    refused(call, **args, workspace=None)
    refused(call, **args, workspace=ws[:need - 1])
    refused(call, **args, workspace=ws[:0])
    for off in (1, 16, 128, 255):
        refused(call, **args, workspace=ws[off:off + need])
    # a workspace that holds one of the matrices
    names = ("x", "w", "bias", "residual", "y", "z") if op == "linear" else ("dy", "z", "x", "w", "dx", "dw", "db")
    room = torch.empty(need + (8 << 20), dtype=torch.uint8, device="cuda")
    for name in names:
        for at in (0, need - 2):
            refused(call, **dict(args, **{name: room.data_ptr() + at}), workspace=room[:need])
    torch.cuda.synchronize()
    for m in (o.y, o.z) if op == "linear" else (o.dx, o.dw, o.db):
        assert torch.equal(m.buffer.view(torch.int16), m.before)      # nothing ran
