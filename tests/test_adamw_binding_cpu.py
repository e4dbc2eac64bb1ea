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
        self.table = [table[i].param for i in range(count)]
        ctypes.cast(out, ctypes.POINTER(ctypes.c_void_p))[0] = 1 << 40
        return ag.AG_OK

    def ag_adamw_step(self, handle, hyper, stream):
        h = hyper._obj
        self.steps.append((h.dev_step, h.dev_lr, h.dev_grad_scale))
        return ag.AG_OK

    def ag_adamw_read_states(self, handle, m, v, stream):
        self.reads.append((list(m), list(v)))
        return ag.AG_OK

    def ag_adamw_destroy(self, handle):
        return ag.AG_OK


class DeviceTensor:
    """What the handle asks of a tensor in device memory."""

    is_cuda, device = True, torch.device("cuda", 0)
    made = 0

    def __init__(self, n, dtype=torch.float32, contiguous=True):
        DeviceTensor.made += 1
        self.n, self.dtype, self.contiguous, self.at = n, dtype, contiguous, (1 << 44) + (DeviceTensor.made << 30)

    def numel(self):
        return self.n

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return self.at


@pytest.fixture
def library(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ag, "lib", lambda: r)
    monkeypatch.setattr(ag, "_lib", r)
    return r


SIZES = [5, 300, 0, 256]


def lists(state8=False, param=torch.bfloat16, master=False):
    d = {"params": [DeviceTensor(n, param) for n in SIZES], "grads": [DeviceTensor(n, param) for n in SIZES],
         "exp_avgs": [DeviceTensor(n, torch.int8 if state8 else torch.float32) for n in SIZES],
         "exp_avg_sqs": [DeviceTensor(n, torch.uint8 if state8 else torch.float32) for n in SIZES]}
    if master:
        d["masters"] = [DeviceTensor(n) for n in SIZES]
    if state8:
        d["exp_avg_scales"], d["exp_avg_sq_scales"] = ([DeviceTensor(-(-n // 256)) for n in SIZES] for _ in range(2))
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
    assert library.table == [t.at for t in d["params"]]
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
