"""The linear layer's and AdamW's refusals and plans without a GPU, and the pins of their oracle."""

import ctypes
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import (BLOCK, act_oracle, adamw8_codes_oracle, adamw_oracle, decode_oracle,
                                  linear_backward_oracle, linear_oracle, random_bits_oracle, slope_oracle)
from tests.linear_util import HUGE, LARGE

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
A = 1 << 44         # a device address; matrices lie 1 GiB apart
GIB = 1 << 30


def status_of(fn, **k):
    try:
        fn(**k)
    except ag.AgError as exc:
        assert exc.message
        return exc.status
    return ag.AG_OK


# ------------------------------------------------------------------ linear

FORWARD = dict(x=A, w=A + GIB, y=A + 2 * GIB, M=1000, N=3584, K=8192, dtype="bf16", act="gelu", bias=A + 3 * GIB,
               residual=A + 4 * GIB, z=A + 5 * GIB, num_cus=256)
BACKWARD = dict(dy=A, x=A + GIB, w=A + 2 * GIB, z=A + 3 * GIB, dx=A + 4 * GIB, dw=A + 5 * GIB, db=A + 6 * GIB, M=1000,
                N=3584, K=8192, dtype="f16", act="silu", num_cus=256)
INVALID, UNSUPPORTED = ag.AG_ERR_INVALID_ARG, ag.AG_ERR_UNSUPPORTED


@pytest.mark.parametrize("over,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(x=A + 1), INVALID), (dict(bias=A + 3 * GIB + 1), INVALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(dtype="f32"), UNSUPPORTED), (dict(dtype=7), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(ldx=8191), INVALID), (dict(ldw=100), INVALID), (dict(ldy=3583), INVALID), (dict(ldr=1), INVALID),
    (dict(ldz=-3584), INVALID),
    (dict(M=1 << 31), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(K=(1 << 20) + 1), UNSUPPORTED),
    (dict(ldx=(1 << 20) + 1), UNSUPPORTED),
    (dict(y=A + 1000), INVALID), (dict(y=A + GIB), INVALID), (dict(z=A + 2 * GIB), INVALID),
    (dict(z=A + 4 * GIB), INVALID), (dict(y=A + 4 * GIB + 2), INVALID), (dict(y=A + 4 * GIB, ldy=3600), INVALID),
    (dict(num_cus=-1), INVALID),
])
def test_plan_linear_rejects(over, status):
    assert status_of(ag.plan_linear, **dict(FORWARD, **over)) == status


@pytest.mark.parametrize("over", [
    dict(), dict(bias=None, residual=None, z=None), dict(y=A + 4 * GIB), dict(x=A + 2, w=A + GIB + 2), dict(ldx=9001),
    dict(M=0, x=None, y=None), dict(N=0, w=None, y=None), dict(K=0, x=None, w=None), dict(M=1, ldx=1 << 40),
    # y's columns beside x's in rows of one buffer
    dict(x=A, ldx=12000, y=A + 8192 * 2, ldy=12000),
])
def test_plan_linear_accepts(over):
    assert status_of(ag.plan_linear, **dict(FORWARD, **over)) == ag.AG_OK


def test_plan_linear_columns_beside_each_other_may_not_cross():
    assert status_of(ag.plan_linear, **dict(FORWARD, x=A, ldx=12000, y=A + 8190 * 2, ldy=12000)) == INVALID
    assert status_of(ag.plan_linear, **dict(FORWARD, x=A + 3600 * 2, ldx=12000, y=A, ldy=12000)) == ag.AG_OK
    assert status_of(ag.plan_linear, **dict(FORWARD, x=A + 4000 * 2, ldx=12000, y=A, ldy=12000)) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(dy=None), INVALID), (dict(z=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(dw_dtype="bf16"), INVALID), (dict(accumulate=2), INVALID), (dict(lddx=1), INVALID), (dict(lddw=8191), INVALID),
    (dict(dw_dtype="f32", dw=A + 5 * GIB + 2), INVALID), (dict(dtype="f32"), UNSUPPORTED),
    (dict(dx=A + 64), INVALID), (dict(dw=A + 4 * GIB), INVALID), (dict(db=A + 5 * GIB), INVALID),
    (dict(dx=A + GIB), INVALID),
])
def test_plan_linear_backward_rejects(over, status):
    assert status_of(ag.plan_linear_backward, **dict(BACKWARD, **over)) == status


@pytest.mark.parametrize("over", [
    dict(), dict(act="none", z=None), dict(dx=None, w=None), dict(dw=None, x=None), dict(db=None), dict(dw_dtype="f32"),
    dict(accumulate=True), dict(dx=None, dw=None, db=None, dy=None, x=None, w=None, z=None), dict(M=0, dy=None, z=None),
])
def test_plan_linear_backward_accepts(over):
    assert status_of(ag.plan_linear_backward, **dict(BACKWARD, **over)) == ag.AG_OK


def test_reserved_fields_and_null_arguments():
    lib = ag.lib()
    p = ag.LinearPlan()
    assert lib.ag_plan_linear(None, 256, ctypes.byref(p)) == INVALID
    assert lib.ag_plan_linear_backward(None, 256, ctypes.byref(p)) == INVALID
    assert lib.ag_linear(None, None, 0, None) == INVALID
    assert lib.ag_linear_backward(None, None, 0, None) == INVALID
    for cls, fn in ((ag.LinearArgs, lib.ag_plan_linear), (ag.LinearBackwardArgs, lib.ag_plan_linear_backward)):
        a = cls(dtype=ag.AG_BF16)
        assert fn(ctypes.byref(a), 256, None) == INVALID
        a.reserved[0] = 1
        assert fn(ctypes.byref(a), 256, ctypes.byref(p)) == INVALID
    a = ag.LinearArgs(x=0, dtype=ag.AG_BF16, M=4, N=4, K=4)
    assert lib.ag_linear(ctypes.byref(a), None, 0, None) == INVALID and "x" in lib.ag_last_error_message().decode()


def test_plan_linear_counts_work_and_workspace():
    p = ag.plan_linear(**FORWARD)
    assert p.flops == 2.0 * 1000 * 3584 * 8192
    assert p.bytes_read == 2 * (1000 * 8192 + 3584 * 8192 + 3584 + 1000 * 3584) and p.bytes_written == 4 * 1000 * 3584
    q = p.product
    assert q.variant == 2 and q.packed == 0 and p.launches == (2 if p.workspace_bytes else 1)
    assert q.full_tiles <= q.n_programs and -(-1000 // q.tile_m) * -(-3584 // q.tile_n) >= q.full_tiles
    few = ag.plan_linear(**dict(FORWARD, M=1))
    assert few.product.variant == 1 and few.workspace_bytes == 0 and few.launches == 1
    # rows off 4-byte alignment are copied, by the tiles alone
    odd = ag.plan_linear(**dict(FORWARD, x=A + 2, ldw=8193))
    assert odd.product.packed == 3 and odd.workspace_bytes >= 2 * (1000 + 3584) * 8192
    assert ag.plan_linear(**dict(FORWARD, M=1, x=A + 2, ldw=8193)).workspace_bytes == 0


def test_plan_linear_backward_counts_work_and_workspace():
    p = ag.plan_linear_backward(**BACKWARD)
    assert p.flops == 4.0 * 1000 * 3584 * 8192 and p.product.variant == 2 and p.product_dw.variant == 2
    assert p.workspace_bytes >= 2 * 1000 * 3584        # dz
    none = ag.plan_linear_backward(**dict(BACKWARD, act="none", z=None, db=None, dw=None, x=None))
    assert none.product_dw.variant == 0 and none.flops == 2.0 * 1000 * 3584 * 8192
    assert none.launches == (2 if none.workspace_bytes else 1)


def test_the_gpu_tests_sizes_reach_every_product_kernel():
    """Tiles, layouts, whole and cut reductions, and the small layers' gradients in one launch (256 CUs)."""
    seen = set()
    for M, N, K in LARGE + HUGE:
        sizes = dict(M=M, N=N, K=K)
        f = ag.plan_linear(**dict(FORWARD, **sizes)).product
        b = ag.plan_linear_backward(**dict(BACKWARD, **sizes))
        one = b.launches == 2 and b.product.tile_m != 0 and b.product_dw.tile_m != 0    # after the slope kernel
        if one:
            seen.add(("in one launch", b.product.tile_m, N >= M))       # which of 256-row tiles' dx and dw goes first
        for form, q in (("y", f),) if one else (("y", f), ("dx", b.product), ("dw", b.product_dw)):
            seen.add((form, q.tile_m, q.tile_n))
            seen.add((form, "cut" if q.splits > 1 else "whole"))
            if q.splits > 1 and q.full_tiles:
                seen.add((form, "whole rounds, then cut"))
    for form in ("y", "dx", "dw"):
        for want in ((256, 256), (128, 128), (256, 128), ("cut",), ("whole",), ("whole rounds, then cut",)):
            assert (form, *want) in seen, (form, want)
    for want in ((128, True), (256, False), (256, True)):
        assert ("in one launch", *want) in seen, want


def test_launches_without_a_device_report_hip_errors():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    f = {k: v for k, v in FORWARD.items() if k != "num_cus"}
    assert status_of(ag.linear, **f) == ag.AG_ERR_HIP
    assert status_of(ag.linear, **dict(f, x=None)) == INVALID           # arguments are checked first
    assert status_of(ag.linear, **dict(f, M=0)) == ag.AG_OK
    assert status_of(ag.plan_linear, **f) == ag.AG_ERR_HIP              # num_cus 0 asks the device


# ------------------------------------------------------------------ AdamW

def tensor(n=1000, at=A, **over):
    fields = dict(param=at, grad=at + GIB, exp_avg=at + 2 * GIB, exp_avg_sq=at + 3 * GIB, n=n)
    fields.update(over)
    return ag.AdamwTensor(**fields)


def create(tensors, param=ag.AG_BF16, grad=ag.AG_BF16, bits=32, count=None):
    h = ctypes.c_void_p()
    table = (ag.AdamwTensor * max(1, len(tensors)))(*tensors)
    return ag.lib().ag_adamw_create(table, len(tensors) if count is None else count, param, grad, bits, ctypes.byref(h))


SCALES = dict(exp_avg_scale=A + 5 * GIB, exp_avg_sq_scale=A + 6 * GIB)


@pytest.mark.parametrize("tensors,more,status", [
    ([tensor()], dict(count=0), INVALID),
    ([tensor()], dict(count=(1 << 20) + 1), INVALID),
    ([tensor()], dict(param=3), INVALID),
    ([tensor()], dict(grad=-1), INVALID),
    ([tensor()], dict(bits=16), INVALID),
    ([tensor(n=-1)], {}, INVALID),
    ([tensor(n=1 << 40)], {}, INVALID),
    ([tensor(param=0)], {}, INVALID),
    ([tensor(grad=None)], {}, INVALID),
    ([tensor(param=A + 1)], {}, INVALID),
    ([tensor(exp_avg=A + 2 * GIB + 2)], {}, INVALID),
    ([tensor()], dict(bits=8), INVALID),                                        # no scales
    ([tensor(**SCALES)], {}, INVALID),                                          # scales of 32-bit states
    ([tensor(master=A + 4 * GIB)], dict(param=ag.AG_F32), UNSUPPORTED),
    ([tensor(master=A + 4 * GIB), tensor(at=A + 8 * GIB)], {}, INVALID),        # one with, one without
    ([tensor(), tensor(at=A + 1024)], {}, INVALID),                             # overlapping parameters
    ([tensor(exp_avg=A)], {}, INVALID),
    ([tensor(grad=A + 998 * 2)], {}, INVALID),
])
def test_adamw_create_rejects(tensors, more, status):
    assert create(tensors, **more) == status


def test_adamw_create_reaches_the_device_with_good_arguments():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    shared = tensor(at=A + 8 * GIB, grad=A + GIB)        # gradients may be shared
    for tensors, more in (([tensor()], {}), ([tensor(**SCALES)], dict(bits=8)), ([tensor(n=0, param=0)], {}),
                          ([tensor(), shared], {})):
        assert create(tensors, **more) == ag.AG_ERR_HIP


def test_adamw_null_handles():
    lib = ag.lib()
    y = ag.AdamwHyper(step=1, eps=1e-8)
    assert lib.ag_adamw_step(None, ctypes.byref(y), None) == INVALID
    assert lib.ag_adamw_read_states(None, None, None, None) == INVALID
    assert lib.ag_adamw_destroy(None) == ag.AG_OK
    assert lib.ag_adamw_create(None, 1, 0, 0, 32, None) == INVALID


# ------------------------------------------------------------------ the oracle's pins

def torch_act(z, act):
    f = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: f.relu(z), "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh"), "silu": lambda: f.silu(z)}[act]()


@pytest.mark.parametrize("act", ACTS)
def test_oracle_layer_and_gradients_against_autograd(act):
    g = np.random.default_rng(1)
    x, w, b, r, dy = (g.standard_normal(s) for s in ((7, 5), (6, 5), (6,), (7, 6), (7, 6)))
    y, z = linear_oracle(x, w, b, act, r)
    tx, tw, tb, tr = (torch.tensor(t, requires_grad=True) for t in (x, w, b, r))
    ty = torch_act(tx @ tw.t() + tb, act) + tr
    assert np.allclose(y, ty.detach().numpy(), rtol=1e-12, atol=1e-12)
    ty.backward(torch.tensor(dy))
    dx, dw, db, _ = linear_backward_oracle(dy, z, x, w, act)
    for got, want in ((dx, tx), (dw, tw), (db, tb), (dy, tr)):
        assert np.allclose(got, want.grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("act", ACTS)
def test_oracle_slope_against_differences(act):
    z = np.linspace(-6, 6, 997)
    h = 1e-5
    want = (act_oracle(z + h, act) - act_oracle(z - h, act)) / (2 * h)
    away = np.abs(z) > 2 * h if act == "relu" else np.ones_like(z, bool)
    assert np.abs(slope_oracle(z, act) - want)[away].max() < 1e-9
    assert slope_oracle(np.zeros(1), "relu")[0] == 0


def test_oracle_adamw_against_torch():
    g = np.random.default_rng(2)
    p = torch.tensor(g.standard_normal(50), requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in (1, 2, 3):
        grad = g.standard_normal(50)
        p.grad = torch.tensor(grad)
        opt.step()
        q, m, v = adamw_oracle(q, grad, m, v, step, 1e-2, 0.8, 0.95, 1e-6, 0.1)
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_oracle_codes_round_trip_and_keep_live_moments():
    g = np.random.default_rng(3)
    m = g.standard_normal(1000) * 10.0 ** g.uniform(-6, 0, 1000)
    v = m * m
    v[10] = 0.0
    for seed in (None, 5):
        cm, ms, cv, vs = adamw8_codes_oracle(m, v, 0, seed)
        assert cm.min() >= -127 and cm.max() <= 127 and cv.min() >= 0 and cv.max() == 255
        assert cv[10] == 0 and (np.delete(cv, 10) >= 1).all()
        back = decode_oracle(cm, ms, 2, 127.0)
        s = np.repeat(ms.astype(np.float64), BLOCK)[:1000]
        step = 0.5 if seed is None else 1.0     # codes lie within so much of the value's place
        place, code = 127 * np.sqrt(np.abs(m) / s), np.abs(cm)
        assert (np.abs(place - code) <= step + 1e-5).all()
        assert np.allclose(127 * np.sqrt(np.abs(back) / s), code, atol=1e-9)
        again = adamw8_codes_oracle(back, decode_oracle(cv, vs, 4, 255.0), 0, None)
        assert np.array_equal(again[0], cm) and np.array_equal(again[2], cv)     # decoded values keep their codes


def test_oracle_random_bits_are_uniform_and_unrelated_between_seeds():
    n = 1 << 16
    at = np.arange(n, dtype=np.uint64)
    a, b = random_bits_oracle(1, at), random_bits_oracle(2, at)
    for bits in (a & np.uint64(0xFFFF), a >> np.uint64(16)):
        count = np.bincount((bits >> np.uint64(8)).astype(np.int64), minlength=256)
        # 256 cells of n/256 expected: chi-square has mean 255, sigma 22.6
        assert ((count - n / 256) ** 2 / (n / 256)).sum() < 255 + 6 * 22.6
    x, y = (t.astype(np.float64) / 2 ** 32 - 0.5 for t in (a, b))
    for shift in range(-3, 4):      # no place of one seed is a shifted place of the next
        assert abs(np.mean(x * np.roll(y, shift))) < 6 / 12 / np.sqrt(n)
    assert abs(np.mean(x[1:] * x[:-1])) < 6 / 12 / np.sqrt(n)


# ------------------------------------------------------------------ the generated code

def _registers(operand):
    """The vector registers that an operand names, e.g. v[4:7] or v9."""
    m = re.fullmatch(r"v\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"v(\d+)", operand)
    return {int(m.group(1))} if m else set()


def unwaited_uses(lines):
    """Instructions that touch a register which an LDS read before them, on some path, may still be writing.

    A read stays in flight until a wait for the LDS counter to reach zero; what is in flight flows along
    branches and into labels.
    """
    starts = sorted({0} | {i for i, ln in enumerate(lines) if ln.endswith(":")} |
                    {i + 1 for i, ln in enumerate(lines) if re.match(r"s_(cbranch|branch|endpgm)", ln)})
    blocks = [(i, j) for i, j in zip(starts, starts[1:] + [len(lines)]) if i < j]
    label = {lines[i][:-1]: k for k, (i, _) in enumerate(blocks) if lines[i].endswith(":")}
    after = []
    for k, (_, j) in enumerate(blocks):
        last = lines[j - 1]
        m = re.match(r"s_c?branch\S*\s+(\S+)", last)
        to = [label[m.group(1)]] if m and m.group(1) in label else []
        if not re.match(r"s_(branch|endpgm)", last) and k + 1 < len(blocks):
            to.append(k + 1)
        after.append(to)

    def walk(k, flying, found):
        flying = set(flying)
        for ln in lines[blocks[k][0]:blocks[k][1]]:
            if ln.startswith("s_waitcnt") and "lgkmcnt(0)" in ln:
                flying.clear()
                continue
            parts = re.split(r"[\s,]+", ln)
            if flying and any(_registers(q) & flying for q in parts[1:]):
                found.append(ln)
            if ln.startswith(("ds_read_b128", "ds_read_b64_tr_b16")):
                flying |= _registers(parts[1])
        return flying

    entry, todo = [set() for _ in blocks], list(range(len(blocks)))
    while todo:
        k = todo.pop()
        out = walk(k, entry[k], [])
        for n in after[k]:
            if not out <= entry[n]:
                entry[n] |= out
                todo.append(n)
    found = []
    for k in range(len(blocks)):
        walk(k, entry[k], found)
    return found


def test_unwaited_uses_sees_a_missing_wait():
    read = ["ds_read_b128 v[4:7], v1", "ds_read_b64_tr_b16 v[8:9], v2 offset:64"]
    use = "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[20:23], a[0:3]"
    assert unwaited_uses(read + [use]) == [use]
    assert unwaited_uses(read + ["v_mov_b32_e32 v30, v9"]) == ["v_mov_b32_e32 v30, v9"]
    assert unwaited_uses(read + ["s_waitcnt lgkmcnt(0)", use]) == []
    assert unwaited_uses(read + ["v_add_u32_e32 v1, v2, v3"]) == []
    # around a loop's back edge, and not past a branch that is always taken
    assert use in unwaited_uses([".L1:", use] + read + ["s_cbranch_scc1 .L1", "s_endpgm"])
    assert unwaited_uses(read + ["s_branch .L2", ".L1:", use, ".L2:", "s_waitcnt lgkmcnt(0)", "s_endpgm"]) == []


@pytest.fixture(scope="module")
def linear_asm(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc = os.path.join(root, "gemm_all_gather_amd", "csrc")
    tmp = tmp_path_factory.mktemp("isa")

    def compile_one(name):
        out = str(tmp / (name + ".s"))
        subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                        "-packed-fp32-ops", f"-I{csrc}", f"-I{os.path.join(root, 'include')}", "--cuda-device-only",
                        "-S", "-o", out, os.path.join(csrc, name + ".hip")], check=True, capture_output=True)
        return open(out).read()

    with ThreadPoolExecutor(2) as pool:
        return "\n".join(pool.map(compile_one, ("ag_linear_forward_bf16", "ag_linear_grads_bf16")))


def test_product_kernels_wait_for_fragments_and_never_spill(linear_asm):
    kernels = re.findall(r"^(_Z\S*ag_linear_(?:gemm|grads)\S*):", linear_asm, re.M)
    assert len(kernels) == 15 + 6 + 3     # 5 activations, 2 gradients in 3 tiles; in turn either way, side by side
    for k in kernels:
        start = linear_asm.index(f"\n{k}:")
        lines = [ln.split(";", 1)[0].strip() for ln in linear_asm[start:linear_asm.index(".section", start)].splitlines()]
        lines = [ln for ln in lines if ln]
        assert sum(ln.startswith("v_mfma") for ln in lines) >= 32, k
        assert sum(ln.startswith("ds_read") for ln in lines) >= 16, k
        assert not unwaited_uses(lines), (k, unwaited_uses(lines)[:3])
        meta = re.search(r"\.amdhsa_kernel " + re.escape(k) + r"\n(.*?)\.end_amdhsa_kernel", linear_asm, re.S).group(1)
        assert re.search(r"private_segment_fixed_size 0\n", meta), k
