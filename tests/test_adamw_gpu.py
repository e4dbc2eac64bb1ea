"""The AdamW step on the GPU against the float64 oracle.

Bounds: a fp32 update of a few operations is off by at most 16 roundings of its terms; 8-bit codes are decided
exactly and have to be equal to the oracle's.
"""

import numpy as np
import pytest
import torch

from gemm_all_gather_amd import binding as ag
from oracle.linear_oracle import BLOCK, adamw8_codes_oracle, adamw_oracle, decode_oracle
from tests.gpu_util import log, require_gpu
from tests.linear_util import HALF_STEP, TINY, TORCH, U32, assert_close, rounded_bound

pytestmark = pytest.mark.gpu

HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 9, 255, 256, 257, 0, 2047, 2048, 2049, 4096, 4097, 10001, 3]


class Tensors:
    """A list of tensors inside NaN-filled flat buffers, `shift` elements off alignment, with the oracle's copy."""

    def __init__(self, sizes, param, grad, state, master, shift=0, seed=1):
        self.sizes, self.param, self.grad, self.state, self.master = sizes, param, grad, state, master
        self.g64 = np.random.default_rng(seed)
        total = sum(sizes) + 64
        self.start = np.concatenate([[0], np.cumsum(sizes)])[:-1] + 32 + shift
        blocks = [-(-n // BLOCK) for n in sizes]
        self.first = np.concatenate([[0], np.cumsum(blocks)])[:-1]
        flat = lambda t: torch.full((total + shift,), float("nan"), dtype=TORCH[t], device="cuda")  # noqa: E731
        self.flats = {"p": flat(param), "g": flat(grad)}
        if master:
            self.flats["master"] = flat("f32")
        if state == 32:
            self.flats["m"], self.flats["v"] = flat("f32"), flat("f32")
        else:
            self.flats["m"] = torch.full((total + shift,), 77, dtype=torch.int8, device="cuda")
            self.flats["v"] = torch.full((total + shift,), 77, dtype=torch.uint8, device="cuda")
            self.flats["ms"] = torch.full((sum(blocks) + 2,), float("nan"), device="cuda")
            self.flats["vs"] = torch.full((sum(blocks) + 2,), float("nan"), device="cuda")
        part = lambda k: [self.flats[k][s:s + n] for s, n in zip(self.start, sizes)]  # noqa: E731
        scale = lambda k: [self.flats[k][1 + f:1 + f + b] for f, b in zip(self.first, blocks)]  # noqa: E731
        self.parts = {k: scale(k) if k in ("ms", "vs") else part(k) for k in self.flats}
        for i, n in enumerate(sizes):
            p = torch.from_numpy(self.g64.standard_normal(n) * 0.5)
            self.parts["p"][i].copy_(p)
            if master:
                self.parts["master"][i].copy_(p)
            for k in ("m", "v", "ms", "vs"):
                if k in self.parts:
                    self.parts[k][i].zero_()
        more = dict(exp_avg_scales=self.parts["ms"], exp_avg_sq_scales=self.parts["vs"]) if state == 8 else {}
        if master:
            more["masters"] = self.parts["master"]
        self.optimizer = ag.AdamW(self.parts["p"], self.parts["g"], self.parts["m"], self.parts["v"], **more)

    def new_gradients(self):
        for t in self.parts["g"]:
            scale = 10.0 ** self.g64.uniform(-4, 0)
            t.copy_(torch.from_numpy(self.g64.standard_normal(t.numel()) * scale *
                                     10.0 ** self.g64.uniform(-3, 0, t.numel())))

    def f64(self, k, i):
        return self.parts[k][i].double().cpu().numpy()

    def moments(self, i):
        if self.state == 32:
            return self.f64("m", i), self.f64("v", i)
        return (decode_oracle(self.f64("m", i), self.f64("ms", i), 2, 127.0),
                decode_oracle(self.f64("v", i), self.f64("vs", i), 4, 255.0))

    def weights(self, i):
        return self.f64("master" if self.master else "p", i)

    def before(self):
        return [(self.weights(i), self.f64("g", i), *self.moments(i)) for i in range(len(self.sizes))]

    def check(self, before, step, what, seed=None, grad_scale=1.0, **hyper):
        torch.cuda.synchronize()
        h = dict(HYPER, **hyper)
        for i, (p, g, m, v) in enumerate(before):
            name = f"{what}, tensor {i} of {self.sizes[i]}"
            p1, m1, v1 = adamw_oracle(p, g, m, v, step, h["lr"], h["beta1"], h["beta2"], h["eps"], h["weight_decay"],
                                      grad_scale)
            gs = np.abs(g * grad_scale)
            m_off = 4 * U32 * (np.abs(h["beta1"] * m) + (1 - h["beta1"]) * gs) + TINY["f32"]
            v_off = 6 * U32 * v1 + TINY["f32"]
            if self.state == 32:
                assert_close(self.f64("m", i), m1, m_off, name + " m")
                assert_close(self.f64("v", i), v1, v_off, name + " v")
            else:
                cm, ms, cv, vs = adamw8_codes_oracle(m1, v1, int(self.first[i]), seed)
                assert np.array_equal(self.f64("ms", i), ms.astype(np.float64)), name + " ms"
                assert np.array_equal(self.f64("vs", i), vs.astype(np.float64)), name + " vs"
                assert np.array_equal(self.f64("m", i), cm), name + " m codes"
                assert np.array_equal(self.f64("v", i), cv), name + " v codes"
            # the step's size: first moment's error through the quotient, the root's and the quotient's roundings
            den = np.sqrt(v1 / (1 - h["beta2"] ** step)) + h["eps"]
            rate = h["lr"] / (1 - h["beta1"] ** step)
            p_off = rate * m_off / den + 16 * U32 * (np.abs(p) + rate * np.abs(m1) / den)
            if self.master:
                assert_close(self.f64("master", i), p1, rounded_bound(p1, p_off, "f32"), name + " master")
            assert_close(self.f64("p", i), p1, rounded_bound(p1, p_off, self.param), name + " p")
        for k, f in self.flats.items():
            used = torch.zeros(f.numel(), dtype=torch.bool, device="cuda")
            at = [1 + int(s) for s in self.first] if k in ("ms", "vs") else [int(s) for s in self.start]
            for s, t in zip(at, self.parts[k]):
                used[s:s + t.numel()] = True
            rest = f[~used]
            assert (torch.isnan(rest).all() if f.is_floating_point() else (rest == 77).all()), f"{what}: {k} written outside"


KINDS = [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "bf16", True), ("f16", "f32", True),
         ("f16", "f16", False), ("bf16", "f32", False), ("f32", "bf16", False)]


@pytest.mark.parametrize("state", [32, 8])
@pytest.mark.parametrize("param,grad,master", KINDS)
def test_adamw_steps(param, grad, master, state):
    require_gpu()
    for shift in (0, 1):
        t = Tensors(SIZES, param, grad, state, master, shift)
        for step in (1, 2, 3):
            t.new_gradients()
            before = t.before()
            seed = None if step == 1 else step if step == 2 else (7 << 40) + 12345
            what = f"adamw {param} {grad} master {master} state {state} shift {shift} step {step}"
            log(what)
            t.optimizer.step(step, **HYPER, seed=seed if state == 8 else None)
            t.check(before, step, what, seed)


def test_adamw_gradient_scale_and_device_scalars():
    require_gpu()
    for state in (32, 8):
        t = Tensors([300, 5000], "bf16", "f16", state, True)
        dev = (torch.tensor([41], device="cuda"), torch.tensor([0.003], device="cuda"), torch.tensor([0.25], device="cuda"))
        t.new_gradients()
        before = t.before()
        log(f"adamw device scalars, state {state}")
        t.optimizer.step(1, **HYPER, grad_scale=0.5, seed=1000 if state == 8 else None, dev_step=dev[0], dev_lr=dev[1],
                         dev_grad_scale=dev[2])
        t.check(before, 41, f"adamw device scalars, state {state}", 1041, 0.125, lr=float(np.float32(0.003)))


def test_adamw_many_tensors():
    require_gpu()
    g = np.random.default_rng(3)
    sizes = [int(n) for n in 10 ** g.uniform(0, 3.5, 500)]
    for state in (32, 8):
        t = Tensors(sizes, "f32", "f32", state, False, 3)
        t.new_gradients()
        before = t.before()
        log(f"adamw 500 tensors, state {state}")
        t.optimizer.step(1, **HYPER)
        t.check(before, 1, f"adamw 500 tensors, state {state}")


def test_adamw_read_states():
    require_gpu()
    sizes = [3, 0, 256, 5001, 0] * 30 + [0]
    t = Tensors(sizes, "f32", "f32", 8, False)
    t.new_gradients()
    t.optimizer.step(1, **HYPER, seed=9)
    out = [[torch.full((n + 2,), float("nan"), device="cuda") for n in sizes] for _ in range(2)]
    log("adamw read states")
    t.optimizer.read_states(*([o[1:-1] for o in part] for part in out))
    torch.cuda.synchronize()
    for i, n in enumerate(sizes):
        for got, want in zip((out[0][i], out[1][i]), t.moments(i)):
            assert torch.isnan(got[0]) and torch.isnan(got[-1])
            assert_close(got[1:-1].double().cpu().numpy(), want, 2 * U32 * np.abs(want) + TINY["f32"], f"tensor {i}")


def test_adamw_beyond_32_bit_offsets():
    """A tensor of more than 2^31 elements: its last block."""
    require_gpu()
    n, last = 2 ** 31 + 5000, 136       # 5000 = 19 blocks and 136 elements
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros_like(p)
    blocks = -(-n // BLOCK)
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(blocks, device="cuda"), torch.zeros(blocks, device="cuda")
    g[-last:] = torch.randn(last, device="cuda").bfloat16()
    opt = ag.AdamW([p], [g], [m], [v], exp_avg_scales=[ms], exp_avg_sq_scales=[vs])
    log("adamw beyond 2^31 elements")
    opt.step(1, **HYPER, seed=11)
    torch.cuda.synchronize()
    g64 = g[-last:].double().cpu().numpy()
    p1, m1, v1 = adamw_oracle(np.zeros(last), g64, np.zeros(last), np.zeros(last), 1, HYPER["lr"], HYPER["beta1"],
                              HYPER["beta2"], HYPER["eps"], HYPER["weight_decay"])
    cm, sm, cv, sv = adamw8_codes_oracle(m1, v1, blocks - 1, 11)
    assert np.array_equal(m[-last:].double().cpu().numpy(), cm) and np.array_equal(v[-last:].double().cpu().numpy(), cv)
    assert ms[-1].item() == sm[0] and vs[-1].item() == sv[0]
    assert_close(p[-last:].double().cpu().numpy(), p1, rounded_bound(p1, 32 * U32 * np.abs(p1), "bf16"), "p")
    assert not p[:-last].any() and not m[:-last].any() and not vs[:-1].any()


def test_adamw_8bit_nothing_live_meets_a_zero_denominator():
    """Gradients a million times smaller than their block's largest still move by at most a few times lr."""
    require_gpu()
    t = Tensors([512], "f32", "f32", 8, False)
    p = t.weights(0)
    t.parts["g"][0].fill_(1e-6)
    t.parts["g"][0][17] = 1.0
    for step in range(1, 6):
        log(f"adamw 8 bit spread, step {step}")
        t.optimizer.step(step, 1e-2, 0.9, 0.99, 1e-12, 0.0, seed=step)
    torch.cuda.synchronize()
    moved = np.abs(t.weights(0) - p)
    assert np.isfinite(moved).all() and moved.max() < 5 * 1e-2 * 10
    assert (t.f64("v", 0) >= 1).all()


@pytest.mark.parametrize("eps", [1e-8, 1e-12, 9e-13, 1e-20])
@pytest.mark.parametrize("state", [32, 8])
def test_adamw_tiny_gradients_and_eps(state, eps):
    """Second moments from 1e-36 (normal in fp32) to 1e-30, whose roots lie far below the larger eps and far above the smallest."""
    require_gpu()
    t = Tensors([1000, 9], "f32", "f32", state, False)
    g = np.random.default_rng(5)
    for step in (1, 2):
        for x in t.parts["g"]:
            n = x.numel()
            x.copy_(torch.from_numpy(g.choice([-1.0, 1.0], n) * 10.0 ** g.uniform(-17, -14, n)))
        before = t.before()
        log(f"adamw tiny gradients, state {state} eps {eps} step {step}")
        t.optimizer.step(step, 1e-2, 0.9, 0.99, eps, 0.1)
        t.check(before, step, f"adamw tiny gradients, state {state} eps {eps} step {step}", eps=eps)


def test_adamw_non_finite_gradients():
    """A NaN or an infinity reaches its own parameter, and its whole block of an 8-bit state; nothing else."""
    require_gpu()
    for bad in (float("nan"), float("inf")):
        for state in (32, 8):
            t = Tensors([1000], "f32", "f32", state, False)
            t.new_gradients()
            t.parts["g"][0][300] = bad
            log(f"adamw {bad} state {state}")
            t.optimizer.step(1, **HYPER)
            torch.cuda.synchronize()
            p, (m, v) = t.weights(0), t.moments(0)
            rest = np.arange(1000) != 300
            assert np.isnan(p[300]) and np.isfinite(p[rest]).all()
            if state == 32:
                assert not np.isfinite(m[300]) and not np.isfinite(v[300])
                assert np.isfinite(m[rest]).all() and np.isfinite(v[rest]).all()
            else:
                block = np.arange(1000) // BLOCK == 300 // BLOCK
                for s in (m, v):
                    assert np.isnan(s[block]).all() and np.isfinite(s[~block]).all()


def test_adamw_stochastic_rounding_is_unbiased():
    """A second moment that decays by 0.1% a step, far below a code's step, decays on average."""
    require_gpu()
    n = 256 * 64
    t = Tensors([n], "f32", "f32", 8, False)
    t.parts["g"][0].fill_(1.0)
    t.parts["g"][0][::256] = 4.0            # every block's maximum
    t.optimizer.step(1, **HYPER)
    start = t.moments(0)[1]
    t.parts["g"][0].zero_()
    t.parts["g"][0][::256] = 4.0 * np.sqrt(0.01)   # the maximum stays: (1 - b2) g^2 of the start
    steps = 100
    for k in range(steps):
        t.optimizer.step(2 + k, 1e-2, 0.9, 0.999, 1e-8, 0.0, seed=1000 + k)
        t.parts["g"][0][::256] = 4.0 * np.sqrt(0.01)
    torch.cuda.synchronize()
    small = np.arange(n) % 256 != 0
    got, want = t.moments(0)[1][small], start[small] * 0.999 ** steps
    # the mean of 16320 independent walks: each of `steps` code steps of under 4/100 with probability under 3%
    sigma = 0.04 * np.sqrt(steps * 0.03) / np.sqrt(small.sum())
    ratio = (got / want).mean()
    assert abs(ratio - 1) < 6 * sigma + 2e-3, ratio
    assert got.std() > 0                   # they walked


def test_adamw_captured_and_replayed():
    require_gpu()
    t = Tensors([1000, 5000], "bf16", "bf16", 8, True)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def call(stream):
        step.add_(1)
        t.optimizer.step(1, **HYPER, seed=50, dev_step=step, stream=stream)

    side = torch.cuda.Stream()
    t.new_gradients()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for rep in range(3):
        t.new_gradients()
        torch.cuda.synchronize()
        before = t.before()
        log(f"adamw graph replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        k = int(step.item())
        assert k == 2 + rep
        t.check(before, k, f"adamw replay {rep}", 50 + k)


def test_bounds_follow_the_types():
    assert HALF_STEP["bf16"] == 2.0 ** -8
