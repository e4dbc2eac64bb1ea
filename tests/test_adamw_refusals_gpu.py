"""AdamW's refusals that need a handle, and so a device: hyper-parameters, outputs, device scalars, destroyed handles.

All of them are found on the host, before a launch.
"""

import ctypes
import math

import pytest
import torch

from gemm_all_gather_amd import binding as ag
from tests.gpu_util import log, require_gpu

pytestmark = pytest.mark.gpu

GOOD = dict(step=1, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, grad_scale=1.0)
NAN, INF = math.nan, math.inf


def make(state8=False, n=300):
    z = lambda d, k=n: torch.zeros(k, dtype=d, device="cuda")  # noqa: E731
    blocks = -(-n // ag.AG_ADAMW_BLOCK)
    states = (z(torch.int8), z(torch.uint8)) if state8 else (z(torch.float32), z(torch.float32))
    more = dict(exp_avg_scales=[z(torch.float32, blocks)], exp_avg_sq_scales=[z(torch.float32, blocks)]) if state8 else {}
    tensors = [torch.ones(n, device="cuda"), torch.ones(n, device="cuda"), *states]
    return tensors, ag.AdamW(*([t] for t in tensors), **more)


@pytest.mark.parametrize("over", [
    dict(step=0), dict(step=-1), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=NAN), dict(beta2=1.0), dict(beta2=-1e-9),
    dict(beta2=NAN), dict(eps=0.0), dict(eps=-1e-8), dict(eps=NAN), dict(eps=INF), dict(eps=1e-60), dict(lr=NAN), dict(lr=INF),
    dict(weight_decay=-INF), dict(weight_decay=NAN), dict(grad_scale=INF), dict(grad_scale=NAN),
])
def test_hyper_parameters_that_are_refused(over):
    require_gpu()
    tensors, opt = make()
    log(f"adamw refuses {over}")
    with pytest.raises(ag.AgError) as exc:
        opt.step(**dict(GOOD, **over))
    assert exc.value.status == ag.AG_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((tensors[0] == 1).all()) and not tensors[2].any()
    opt.destroy()


def test_reserved_fields_and_flags_are_refused():
    require_gpu()
    _, opt = make()
    lib = ag.lib()
    log("adamw refuses reserved fields and flags")
    y = lambda **k: ag.AdamwHyper(1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0, 1, **k)  # noqa: E731
    h = y()
    h.reserved[4] = 1
    for bad in (h, y(stochastic=2), y(stochastic=-1)):
        assert lib.ag_adamw_step(opt.handle, ctypes.byref(bad), None) == ag.AG_ERR_INVALID_ARG
    assert lib.ag_adamw_step(opt.handle, None, None) == ag.AG_ERR_INVALID_ARG
    opt.destroy()
    with pytest.raises(RuntimeError):
        opt.step(**GOOD)


def test_reading_states_that_are_refused():
    require_gpu()
    out = lambda: torch.empty(300, device="cuda")  # noqa: E731
    _, opt = make()
    log("adamw refuses outputs of read_states")
    with pytest.raises(ag.AgError) as exc:      # fp32 states are what they are
        opt.read_states([out()], [out()])
    assert exc.value.status == ag.AG_ERR_INVALID_ARG
    opt.destroy()
    _, opt = make(True)
    for bad in (out()[:299], out().half(), torch.empty(600, device="cuda")[::2], torch.empty(300)):
        for pair in ((bad, out()), (out(), bad)):
            with pytest.raises(ValueError):
                opt.read_states(*([t] for t in pair))
    a = out()
    for pair in ((a.data_ptr() + 2, out()), (out(), 0)):        # an address off fp32's alignment, and none
        with pytest.raises(ag.AgError):
            opt.read_states(*([t] for t in pair))
    m, v = out(), out()
    opt.read_states([m], [v])
    torch.cuda.synchronize()
    assert not m.any() and not v.any()
    opt.destroy()


def test_host_memory_is_refused_and_pinned_memory_is_not():
    require_gpu()
    host = torch.zeros(300)
    dev = lambda: torch.zeros(300, device="cuda")  # noqa: E731
    log("adamw refuses host memory")
    for i in range(4):
        tensors = [[host if i == k else dev()] for k in range(4)]
        with pytest.raises(ValueError):
            ag.AdamW(*tensors)
    _, opt = make()
    with pytest.raises(ValueError):
        opt.step(**GOOD, dev_step=torch.ones(1, dtype=torch.int64))
    opt.destroy()
    log("adamw with pinned states")
    m, v = (torch.zeros(300, pin_memory=True) for _ in range(2))
    p = torch.ones(300, device="cuda")
    opt = ag.AdamW([p], [torch.ones(300, device="cuda")], [m], [v])
    opt.step(**GOOD)
    torch.cuda.synchronize()
    assert torch.allclose(m, torch.full((300,), 0.1)) and bool((p < 1).all())
    opt.destroy()


def test_a_step_after_the_callers_lists_have_changed():
    require_gpu()
    n = 300
    make_list = lambda v: [torch.full((n,), v, device="cuda")]  # noqa: E731
    params, grads, m, v = make_list(1.0), make_list(2.0), make_list(0.0), make_list(0.0)
    kept = params[0], m[0]
    opt = ag.AdamW(params, grads, m, v)
    grads.clear()
    m[0] = v[0] = params[0] = None
    torch.cuda.synchronize()
    other = [torch.full((n,), float("nan"), device="cuda") for _ in range(8)]       # would take freed tensors' memory
    log("adamw after its lists have changed")
    opt.step(**GOOD)
    torch.cuda.synchronize()
    assert torch.allclose(kept[1], torch.full_like(kept[1], 0.2)) and bool(torch.isfinite(kept[0]).all())
    assert all(bool(torch.isnan(t).all()) for t in other)
    opt.destroy()
