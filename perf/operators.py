"""Measured cases of the layer operators: the linear layer with its epilogue, its gradients, and the AdamW step.

The plain forms here are elementary torch operations in 32 bits (64 where codes of 8 bits are decided); with
``own`` set the same work goes through the library's entry points in gemm_all_gather_amd.binding.
"""

import itertools
import math

import torch

own = False

BLOCK = 256                 # elements of one block of 8-bit states
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ADAM = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1}
FIRST_STEP = 100            # steps taken before the measured one


def _linear(name, M, N, K, dtype, act, bias, residual, save, pad=0):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save": save, "pad": pad}


def _backward(name, M, N, K, dtype, act, bias, dw, accumulate, pad=0):
    return {"name": name, "op": "backward", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias,
            "dw": dw, "accumulate": accumulate, "pad": pad}


def _adamw(name, tensors, rows, cols, state, param, grad, master, packed):
    return {"name": name, "op": "adamw", "tensors": tensors, "rows": rows, "cols": cols, "state": state,
            "param": param, "grad": grad, "master": master, "packed": packed}


def listed():
    return [
        # one token through a layer, as in serving: the weights are streamed once
        _linear("decode 1", 1, 3584, 8192, "bf16", "silu", True, False, False),
        # a few sequences decoded together, the second product of a block with its residual
        _linear("decode 13", 13, 8192, 3584, "f16", "none", True, True, False),
        # a short prompt
        _linear("prompt 1024", 1024, 3584, 8192, "bf16", "gelu", True, True, False),
        # a training micro-batch, the pre-activation kept for the backward pass
        _linear("train 16384", 16384, 3584, 8192, "bf16", "gelu_tanh", True, False, True),
        # sizes that are no multiple of a tile or of a 16-byte vector
        _linear("ragged 1000", 1000, 4100, 4100, "f16", "relu", True, True, False),
        # gradients of a small layer: latency
        _backward("backward 80", 80, 520, 136, "f16", "relu", True, "f16", False),
        # gradients of a short micro-batch
        _backward("backward 1024", 1024, 3584, 8192, "bf16", "gelu", True, "bf16", False),
        # gradients of the training micro-batch
        _backward("backward 16384", 16384, 3584, 8192, "bf16", "gelu_tanh", True, "bf16", False),
        # ragged, the weight gradient added up in 32 bits over micro-batches
        _backward("backward ragged", 1000, 4100, 4100, "bf16", "none", True, "f32", True),
        # four weights and their biases, master weights and states in 32 bits
        _adamw("adamw 32 bit", 4, 3584, 8192, 32, "bf16", "bf16", True, False),
        # the same with states in 8 bits, and no master weights
        _adamw("adamw 8 bit", 4, 3584, 8192, 8, "bf16", "bf16", False, False),
        # a model's many small tensors, tightly packed
        _adamw("adamw small", 300, 1, 16384, 32, "f32", "f32", False, True),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 37 if n // 64 == 48 else n


def draw(rng):
    op = rng.choice(("linear", "linear", "backward", "backward", "adamw"))
    if op == "adamw":
        state = rng.choice((32, 8))
        param = rng.choice(("bf16", "f16", "f32"))
        tensors = _log(rng, 1, 400)
        largest = _log(rng, 256, min(3584 * 8192, 4 * 3584 * 8192 // tensors))
        rows = rng.choice((1, 1, _log(rng, 1, 64)))
        return _unnamed(_adamw("", tensors, rows, max(1, largest // rows), state, param,
                               rng.choice((param, "f32")), param != "f32" and rng.random() < 0.5,
                               state == 32 and rng.random() < 0.5))
    M, N, K = _log(rng, 1, 16384), _log(rng, 64, 8192), _log(rng, 64, 8192)
    if rng.random() < 0.5:      # half of them in whole vectors, as most models have them
        N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
    while 2.0 * M * N * K > 2.0 * 16384 * 3584 * 8192:
        M = max(1, M // 2)
    dtype, act = rng.choice(("bf16", "f16")), rng.choice(ACTS)
    pad = rng.choice((0, 0, 8, 3))
    if op == "linear":
        return _unnamed(_linear("", M, N, K, dtype, act, rng.random() < 0.7, rng.random() < 0.5,
                                rng.random() < 0.5, pad))
    # a weight gradient kept in 32 bits is drawn where no activation rounds dz to 16 bits first
    dw = "f32" if act == "none" and rng.random() < 0.5 else dtype
    return _unnamed(_backward("", M, N, K, dtype, act, rng.random() < 0.7, dw, rng.random() < 0.3, pad))


def _unnamed(case):
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _randn(gen, rows, cols, pad, dtype, scale=1.0):
    """A rows x cols matrix whose rows are cols + pad elements apart."""
    full = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32)
    return full.mul_(scale).to(dtype)[:, :cols]


def _sizes(case):
    """The elements of each tensor: weights and their biases, or sizes spread from 1 to rows*cols."""
    n, largest = case["tensors"], case["rows"] * case["cols"]
    if n <= 8:
        return [size for _ in range(n) for size in (largest, case["rows"])]
    return [max(1, int(largest ** ((i * 0.6180339887) % 1.0))) for i in range(1, n + 1)]


def _hash(seed, count, device):
    """The stochastic rounding's 32 random bits of state element i (in 64-bit integers)."""
    whole, low = (1 << 64) - 1, 0xFFFFFFFF
    z = seed + 0x9E3779B97F4A7C15 & whole
    z = (z ^ z >> 30) * 0xBF58476D1CE4E5B9 & whole
    z = (z ^ z >> 27) * 0x94D049BB133111EB & whole
    z ^= z >> 31
    i = torch.arange(count, device=device, dtype=torch.int64)
    x = (i & low) ^ ((z & low) + (i >> 32) * 0x9E3779B1 & low)
    x = (x ^ x >> 16) * 0x7FEB352D & low
    x = (x ^ x >> 15) ^ z >> 32
    x = x * 0x846CA68B & low
    return x ^ x >> 16


def _encode(value, power, top, u):
    """Codes and block maxima of non-negative values in 64 bits: value = (code/top)^power * maximum."""
    v = value.view(-1, BLOCK)
    s = v.amax(1, keepdim=True).to(torch.float32)
    sd = s.double()
    t = (v / torch.where(sd > 0, sd, 1.0)).pow(1.0 / power) * top
    c = torch.where(sd > 0, torch.floor(t + u.view(-1, BLOCK)).clamp_(0, top), 0.0)
    return c, s


def _offsets(uniform32):
    """The two offsets in (0, 1) that an element's random bits give its two codes."""
    return ((uniform32 & 0xFFFF).double() + 0.5) / 65536, ((uniform32 >> 16).double() + 0.5) / 65536


def _prepare_adamw(case, gen):
    sizes = _sizes(case)
    step = [n if case["packed"] else -(-n // BLOCK) * BLOCK for n in sizes]
    total = sum(step)
    # the tensors are views of flat buffers, as sharded training keeps them
    p = torch.randn(total, generator=gen, device="cuda") * 0.02
    g = torch.randn(total, generator=gen, device="cuda") * 0.01
    m = torch.randn(total, generator=gen, device="cuda") * 0.003
    v = torch.rand(total, generator=gen, device="cuda") ** 2 * 3e-4 + m * m
    starts = [0] + list(itertools.accumulate(step))[:-1]
    each = lambda t: torch.repeat_interleave(torch.tensor(t, device="cuda"), torch.tensor(step, device="cuda"))  # noqa: E731
    gap = torch.arange(total, device="cuda") - each(starts) >= each(sizes)      # between tensors
    p, g, m, v = (t.masked_fill_(gap, 0.0) for t in (p, g, m, v))
    s = {"step": FIRST_STEP, "p": p.to(TYPES[case["param"]]), "g": g.to(TYPES[case["grad"]])}
    if case["master"]:
        s["master"] = p
    if case["state"] == 32:
        s["m"], s["v"] = m, v
    else:
        half = torch.full((total,), 0.5, device="cuda", dtype=torch.float64)
        c, s["ms"] = _encode(m.double().abs(), 2, 127.0, half)
        s["m"] = (c * m.view(-1, BLOCK).sign()).to(torch.int8).view(-1)
        c, s["vs"] = _encode(v.double(), 4, 255.0, half)
        s["v"] = torch.where(v.view(-1, BLOCK) > 0, c.clamp_(min=1), c).to(torch.uint8).view(-1)
        s["ms"], s["vs"] = s["ms"].view(-1), s["vs"].view(-1)
        s["m_read"], s["v_read"] = torch.zeros_like(p), torch.zeros_like(p)
    if own:
        from gemm_all_gather_amd import binding as ag
        parts = lambda t: [t[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
        scales = lambda t: [t[a // BLOCK:(a + n + BLOCK - 1) // BLOCK] for a, n in zip(starts, sizes)]  # noqa: E731
        more = {"masters": parts(s["master"])} if case["master"] else {}
        if case["state"] == 8:
            more.update(exp_avg_scales=scales(s["ms"]), exp_avg_sq_scales=scales(s["vs"]))
            s["reads"] = parts(s["m_read"]), parts(s["v_read"])
        s["optimizer"] = ag.AdamW(parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]), **more)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "adamw":
        s.update(_prepare_adamw(case, gen))
        return s
    M, N, K, pad, dt = case["M"], case["N"], case["K"], case["pad"], TYPES[case["dtype"]]
    s["x"] = _randn(gen, M, K, pad, dt)
    s["w"] = _randn(gen, N, K, pad, dt, 1.0 / math.sqrt(K))
    empty = lambda rows, cols, t: torch.empty(rows, cols + pad, device="cuda", dtype=t)[:, :cols]  # noqa: E731
    if case["op"] == "linear":
        s["b"] = _randn(gen, 1, N, 0, dt, 0.1)[0] if case["bias"] else None
        s["r"] = _randn(gen, M, N, pad, dt) if case["residual"] else None
        s["y"] = empty(M, N, dt)
        s["z"] = empty(M, N, dt) if case["save"] else None
    else:
        s["dy"] = _randn(gen, M, N, pad, dt)
        s["z"] = _randn(gen, M, N, pad, dt) if case["act"] != "none" else None
        s["dx"], s["dw"] = empty(M, K, dt), empty(N, K, TYPES[case["dw"]])
        s["db"] = torch.empty(N, device="cuda", dtype=TYPES[case["dw"]]) if case["bias"] else None
        if case["accumulate"]:      # what the micro-batches before this one added up
            s["dw"].copy_(_randn(gen, N, K, pad, TYPES[case["dw"]]))
            if case["bias"]:
                s["db"].copy_(_randn(gen, 1, N, 0, TYPES[case["dw"]])[0])
    if own:
        from gemm_all_gather_amd import binding as ag
        plan = ag.plan_linear if case["op"] == "linear" else ag.plan_linear_backward
        s["workspace"] = torch.empty(max(1, plan(**_arguments(s)).workspace_bytes), device="cuda", dtype=torch.uint8)
    return s


def _arguments(s):
    """The keyword arguments of the library's linear and linear_backward."""
    c = s["case"]
    a = {"M": c["M"], "N": c["N"], "K": c["K"], "dtype": c["dtype"], "act": c["act"], "x": s["x"], "w": s["w"],
         "z": s["z"], "ldx": s["x"].stride(0), "ldw": s["w"].stride(0)}
    if s["z"] is not None:
        a["ldz"] = s["z"].stride(0)
    if c["op"] == "linear":
        a.update(bias=s["b"], residual=s["r"], y=s["y"], ldy=s["y"].stride(0))
        if s["r"] is not None:
            a["ldr"] = s["r"].stride(0)
    else:
        a.update(dy=s["dy"], lddy=s["dy"].stride(0), dx=s["dx"], lddx=s["dx"].stride(0), dw=s["dw"],
                 lddw=s["dw"].stride(0), db=s["db"], dw_dtype=c["dw"], accumulate=c["accumulate"])
    return a


# ------------------------------------------------------------------ the plain forms

def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, 0.0, z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return torch.where(z <= 0, 0.0, 1.0)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * z * z)
    e = torch.exp(-z)
    return (1.0 + e + z * e) / ((1.0 + e) * (1.0 + e))


def _plain_linear(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    z = s["x"].float() @ s["w"].float().t()
    if c["bias"]:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["r"].float()
    return [y.to(dt)] + ([z.to(dt)] if c["save"] else [])


def _plain_backward(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), c["act"])
    dx = dz @ s["w"].float()
    dw = dz.t() @ s["x"].float()
    db = dz.double().sum(0).float() if c["bias"] else None
    if c["accumulate"]:
        dw = dw + s["dw"].float()
        db = db + s["db"].float() if c["bias"] else None
    s["dw"].copy_(dw)
    if c["bias"]:
        s["db"].copy_(db)
    return [dx.to(dt), s["dw"]] + ([s["db"]] if c["bias"] else [])


def _plain_adamw(s):
    a, c = ADAM, s["case"]
    bc1, bc2 = 1.0 - a["beta1"] ** s["step"], 1.0 - a["beta2"] ** s["step"]
    p = (s["master"] if c["master"] else s["p"]).float()
    if c["state"] == 32:
        g = s["g"].float()
        m, v = s["m"], s["v"]
        m.mul_(a["beta1"]).add_(g, alpha=1.0 - a["beta1"])
        v.mul_(a["beta2"]).add_(g * g, alpha=1.0 - a["beta2"])
        out = [m, v]
    else:               # the codes are decided in 64 bits: a value next to a border takes the same side everywhere
        g = s["g"].double()
        c8, ms, vs = s["m"].double(), s["ms"].double(), s["vs"].double()
        m = (c8 * c8.abs()).view(-1, BLOCK) * (ms * (1.0 / 127.0 ** 2)).view(-1, 1)
        m = a["beta1"] * m.view(-1) + (1.0 - a["beta1"]) * g
        v = s["v"].double().pow(4).view(-1, BLOCK) * (vs * (1.0 / 255.0 ** 4)).view(-1, 1)
        v = a["beta2"] * v.view(-1) + (1.0 - a["beta2"]) * g * g
        um, uv = _offsets(_hash(s["step"], m.numel(), m.device))
        cm, ms = _encode(m.abs(), 2, 127.0, um)
        cv, vs = _encode(v, 4, 255.0, uv)
        cm, cv = cm * m.view(-1, BLOCK).sign(), torch.where(v.view(-1, BLOCK) > 0, cv.clamp(min=1), cv)
        s["m"].copy_(cm.view(-1))
        s["v"].copy_(cv.view(-1))
        s["ms"].copy_(ms.view(-1))
        s["vs"].copy_(vs.view(-1))
        out = [(cm * cm.abs() * (ms.double() * (1.0 / 127.0 ** 2))).float().view(-1),
               (cv.pow(4) * (vs.double() * (1.0 / 255.0 ** 4))).float().view(-1)]
        m, v = m.float(), v.float()
    p = p * (1.0 - a["lr"] * a["weight_decay"]) - a["lr"] * (m / bc1) / ((v / bc2).sqrt() + a["eps"])
    s["p"].copy_(p)
    if c["master"]:
        s["master"].copy_(p)
    return [s["p"]] + ([s["master"]] if c["master"] else []) + out


def run(s):
    op = s["case"]["op"]
    if op == "adamw":
        s["step"] += 1
    if not own:
        return {"linear": _plain_linear, "backward": _plain_backward, "adamw": _plain_adamw}[op](s)
    from gemm_all_gather_amd import binding as ag
    stream = torch.cuda.current_stream()
    if op == "adamw":
        opt, a, c = s["optimizer"], ADAM, s["case"]
        opt.step(s["step"], a["lr"], a["beta1"], a["beta2"], a["eps"], a["weight_decay"],
                 seed=s["step"] if c["state"] == 8 else None, stream=stream)
        if c["state"] == 8:     # the values that the codes stand for, as a checkpoint takes them
            opt.read_states(*s["reads"], stream=stream)
        out = [s["m"], s["v"]] if c["state"] == 32 else [s["m_read"], s["v_read"]]
        return [s["p"]] + ([s["master"]] if c["master"] else []) + out
    if op == "linear":
        ag.linear(**_arguments(s), workspace=s["workspace"], stream=stream)
        return [t for t in (s["y"], s["z"]) if t is not None]
    ag.linear_backward(**_arguments(s), workspace=s["workspace"], stream=stream)
    return [t for t in (s["dx"], s["dw"], s["db"]) if t is not None]


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    if case["op"] == "linear":
        z = torch.matmul(f(s["x"]), f(s["w"]).transpose(0, 1).contiguous())
        if s["b"] is not None:
            z += f(s["b"])[None, :]
        y = {"none": lambda: z, "relu": lambda: z.clamp(min=0.0),
             "gelu": lambda: z * torch.special.ndtr(z),
             "gelu_tanh": lambda: z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)),
             "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        if s["r"] is not None:
            y = y + f(s["r"])
        return [y, z] if case["save"] else [y]
    dz = f(s["dy"])
    if case["act"] != "none":
        z = f(s["z"])
        sig = torch.sigmoid(z)
        u = 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z ** 2)
        slope = {"relu": lambda: (z > 0).double(),
                 "gelu": lambda: torch.special.ndtr(z) + z * torch.exp(-z * z / 2.0) * (2.0 * math.pi) ** -0.5,
                 "gelu_tanh": lambda: torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * du,
                 "silu": lambda: sig + z * sig * (1.0 - sig)}[case["act"]]()
        dz = dz * slope
    out = [torch.matmul(dz, f(s["w"])), torch.matmul(dz.transpose(0, 1).contiguous(), f(s["x"]))]
    if case["bias"]:
        out.append(torch.sum(dz, dim=0))
    if case["accumulate"]:
        out[1] += f(s["dw"])
        if case["bias"]:
            out[2] += f(s["db"])
    return out


def _exact_adamw(case, s):
    lr, b1, b2, eps, wd = (ADAM[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    k = FIRST_STEP + 1
    p = (s["master"] if case["master"] else s["p"]).to(torch.float64)
    g, m, v = (s[n].to(torch.float64) for n in ("g", "m", "v"))
    if case["state"] == 8:
        m = torch.sign(m) * (m / 127.0) ** 2 * s["ms"].double().repeat_interleave(BLOCK)
        v = (v / 255.0) ** 4 * s["vs"].double().repeat_interleave(BLOCK)
    m = m + (1.0 - b1) * (g - m)
    v = v + (1.0 - b2) * (g * g - v)
    p = p - lr * wd * p - lr * (m / (1.0 - b1 ** k)) / (torch.sqrt(v / (1.0 - b2 ** k)) + eps)
    if case["state"] == 8:
        bits = _hash(k, m.numel(), m.device)
        m = _rounded(m, 0.5, 127, bits & 0xFFFF, False)
        v = _rounded(v, 0.25, 255, bits >> 16, True)
    return [p, p, m, v] if case["master"] else [p, m, v]


def _rounded(value, root, top, bits, live):
    """Each value as its block's nearest lower or upper code stands for it, by the random bits."""
    size = torch.abs(value).reshape(-1, BLOCK)
    most = torch.max(size, dim=1, keepdim=True).values.float().double()
    place = top * torch.exp(root * torch.log(size / most))         # -inf where a value is zero
    code = torch.floor(torch.nan_to_num(place) + (bits.double() * 2 + 1).reshape(-1, BLOCK) / 131072)
    code = torch.clamp(code, max=top)
    if live:
        code = torch.where(size > 0, torch.clamp(code, min=1), code)
    back = torch.where(most > 0, most * (code / top) ** (1.0 / root), 0.0)
    return torch.sign(value) * back.reshape(-1)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        size = {"bf16": 2, "f16": 2, "f32": 4}
        each = size[case["param"]] + size[case["grad"]]                      # written, and read
        each += 8 if case["master"] else size[case["param"]]                 # master both ways, or the parameter read
        each += 16 if case["state"] == 32 else 4 + 16 / BLOCK + 8            # with the values in 32 bits written
        return {"bytes": n * each, "flops": 14.0 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "linear":
        outs = 1 + case["residual"] + case["save"]
        return {"bytes": 2.0 * (M * K + N * K + outs * M * N + (N if case["bias"] else 0)), "flops": 2.0 * M * N * K}
    d = 4 if case["dw"] == "f32" else 2
    reads = M * N * (2 if case["act"] != "none" else 1) + M * K + N * K
    grads = (N * K + (N if case["bias"] else 0)) * (2 if case["accumulate"] else 1)
    return {"bytes": 2.0 * (reads + M * K) + d * grads, "flops": 4.0 * M * N * K}
