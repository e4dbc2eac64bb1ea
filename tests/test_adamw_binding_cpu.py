"""AdamW's Python handle without a GPU: what it keeps alive and what it refuses before an address reaches the library."""

import ctypes
import gc
import weakref

import pytest
import torch

from gemm_all_gather_amd import binding as ag


class Recorder:
    """Stands in for the library: takes every call, and keeps the addresses it was given."""

    def __init__(self):
        self.table, self.steps, self.reads = [], [], []

    def ag_adamw_create(self, table, count, param, grad, bits, out):
        self.table = [table[i].param or 0 for i in range(count)]
        ctypes.cast(out, ctypes.POINTER(ctypes.c_void_p))[0] = 1 << 40
        return ag.AG_OK

    def ag_adamw_step(self, handle, hyper, stream):
        h = hyper._obj
        self.steps.append((h.dev_step, h.dev_lr, h.dev_grad_scale))
        return ag.AG_OK

    def ag_adamw_read_states(self, handle, m, v, stream):
        self.reads.append(tuple([p or 0 for p in part] for part in (m, v)))      # ctypes gives None for 0
        return ag.AG_OK

    def ag_adamw_destroy(self, handle):
        return ag.AG_OK


def tensor(n, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype)


@pytest.fixture
def library(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ag, "_reachable", lambda tensors: True, raising=False)      # its tensors lie in host memory here
    monkeypatch.setattr(ag, "lib", lambda: r)
    monkeypatch.setattr(ag, "_lib", r)
    return r


SIZES = [5, 300, 0, 256]


def lists(state8=False, param=torch.bfloat16, master=False):
    d = {"params": [tensor(n, param) for n in SIZES], "grads": [tensor(n, param) for n in SIZES],
         "exp_avgs": [tensor(n, torch.int8 if state8 else torch.float32) for n in SIZES],
         "exp_avg_sqs": [tensor(n, torch.uint8 if state8 else torch.float32) for n in SIZES]}
    if master:
        d["masters"] = [tensor(n) for n in SIZES]
    if state8:
        d["exp_avg_scales"], d["exp_avg_sq_scales"] = ([tensor(-(-n // 256)) for n in SIZES] for _ in range(2))
    return d


# ------------------------------------------------------------------ what is kept

def test_tensors_outlive_the_callers_lists(library):
    d = lists(True, master=True)
    opt = ag.AdamW(**d)
    held = [weakref.ref(t) for part in d.values() for t in part]
    for k, part in enumerate(d.values()):
        if k % 2:
            part.clear()
        else:
            part[:] = [None] * len(part)
    gc.collect()
    assert all(r() is not None for r in held)
    opt.destroy()


def test_lists_may_be_any_iterables(library):
    d = lists(True, master=True)
    opt = ag.AdamW(**{k: iter(part) for k, part in d.items()})
    assert library.table == [t.data_ptr() for t in d["params"]]
    opt.destroy()


def test_lists_of_other_lengths_are_refused(library):
    for k in lists(True, master=True):
        d = lists(True, master=True)
        d[k] = d[k][:-1]
        with pytest.raises(ValueError):
            ag.AdamW(**d)
        d[k] = []
        with pytest.raises(ValueError):
            ag.AdamW(**d)


# ------------------------------------------------------------------ outputs of read_states

def outputs():
    return [[tensor(n) for n in SIZES] for _ in range(2)]


def test_read_states_takes_whole_contiguous_fp32_outputs(library):
    opt = ag.AdamW(**lists(True))
    m, v = outputs()
    opt.read_states(m, iter(v))
    assert library.reads == [([t.data_ptr() for t in m], [t.data_ptr() for t in v])]
    addresses = [[t.data_ptr() for t in part] for part in (m, v)]        # addresses go through as they are
    opt.read_states(*addresses)
    assert library.reads[1] == library.reads[0]
    opt.destroy()


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("bad", [lambda: tensor(299), lambda: tensor(301), lambda: tensor(300, torch.float16),
                                 lambda: tensor(300, torch.float64), lambda: tensor(600)[::2]])
def test_read_states_refuses_outputs_it_would_write_past(library, bad, which):
    opt = ag.AdamW(**lists(True))
    out = outputs()
    out[which][1] = bad()
    with pytest.raises(ValueError):
        opt.read_states(*out)
    assert not library.reads
    opt.destroy()


def test_read_states_refuses_lists_of_other_lengths(library):
    opt = ag.AdamW(**lists(True))
    for k in (0, 1):
        for change in (lambda t: t[:-1], lambda t: t + [tensor(1)], lambda t: []):
            out = outputs()
            out[k] = change(out[k])
            with pytest.raises(ValueError):
                opt.read_states(*out)
    assert not library.reads
    opt.destroy()


# ------------------------------------------------------------------ device scalars of a step

def test_step_takes_device_scalars_of_their_types(library):
    opt = ag.AdamW(**lists())
    step, lr, scale = torch.ones(1, dtype=torch.int64), torch.ones(()), torch.ones(3)[1:2]
    opt.step(1, 1e-3, dev_step=step, dev_lr=lr, dev_grad_scale=scale)
    opt.step(1, 1e-3, dev_step=1 << 44, dev_lr=2 << 44)                  # addresses go through as they are
    opt.step(1, 1e-3)
    assert library.steps == [(step.data_ptr(), lr.data_ptr(), scale.data_ptr()), (1 << 44, 2 << 44, None), (None, None, None)]
    opt.destroy()


@pytest.mark.parametrize("name,bad", [
    ("dev_step", torch.ones(1, dtype=torch.int32)), ("dev_step", torch.ones(1)), ("dev_step", torch.ones(0, dtype=torch.int64)),
    ("dev_lr", torch.ones(1, dtype=torch.float64)), ("dev_lr", torch.ones(1, dtype=torch.bfloat16)), ("dev_lr", torch.ones(0)),
    ("dev_grad_scale", torch.ones(1, dtype=torch.float64)), ("dev_grad_scale", torch.ones(1, dtype=torch.int64)),
    ("dev_grad_scale", torch.ones(0)),
])
def test_step_refuses_device_scalars_it_would_misread(library, name, bad):
    opt = ag.AdamW(**lists())
    with pytest.raises(ValueError, match=name):
        opt.step(1, 1e-3, **{name: bad})
    assert not library.steps
    opt.destroy()


# ------------------------------------------------------------------ memory that kernels cannot reach

@pytest.fixture
def strict(library, monkeypatch):
    monkeypatch.undo()                      # the real check of where tensors lie
    r = Recorder()
    monkeypatch.setattr(ag, "lib", lambda: r)
    monkeypatch.setattr(ag, "_lib", r)
    return r


def test_tensors_in_pageable_host_memory_are_refused(strict):
    with pytest.raises(ValueError, match="host memory"):
        ag.AdamW(**lists(True, master=True))
    assert not strict.table
    # tensors without elements have no memory to reach
    opt = ag.AdamW(*([torch.zeros(0)] for _ in range(4)))
    with pytest.raises(ValueError, match="host memory"):
        opt.step(1, 1e-3, dev_lr=torch.ones(1))
    assert not strict.steps
    opt.destroy()


def test_read_states_refuses_host_outputs(library, monkeypatch):
    opt = ag.AdamW(**lists(True))
    monkeypatch.setattr(ag, "_reachable", lambda tensors: False)
    with pytest.raises(ValueError, match="host memory"):
        opt.read_states(*outputs())
    assert not library.reads
    opt.destroy()


def test_reachable_memory():
    class Pinned(torch.Tensor):
        def is_pinned(self):
            return True

    host, pinned = torch.zeros(3), torch.zeros(3).as_subclass(Pinned)
    assert ag._reachable([]) and ag._reachable([torch.zeros(0)]) and ag._reachable([pinned])
    assert not ag._reachable([host]) and not ag._reachable([pinned, host]) and not ag._reachable([torch.zeros(3, device="meta")])


def test_read_states_takes_addresses_among_tensors(library):
    opt = ag.AdamW(**lists(True))
    m, v = outputs()
    want = [t.data_ptr() for t in m], [t.data_ptr() for t in v]
    m[1], v[3] = want[0][1], want[1][3]
    opt.read_states(m, v)
    assert library.reads == [want]
    m[0] = tensor(4)
    with pytest.raises(ValueError):
        opt.read_states(m, v)
    opt.destroy()
