"""Measured cases of the operators around 8-bit activations: the root-mean-square norm with the residual's addition and an
output in 8 bits, its gradients, the linear layer on 8-bit integers, and activation checkpoints in 8 bits with the gradients
that read them.

The plain forms here are elementary torch operations in 32 bits (64 where codes of 8 bits are decided, and in sums over
many rows); with ``own`` set the same work goes through the library's entry points in gemm_all_gather_amd.binding.
"""

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _norm(name, M, K, dtype, residual, out, pad=0):
    """out: "y" (rounded, with the root's reciprocal for the backward pass) or "q8" (codes and a scale for each row)."""
    return {"name": name, "op": "norm", "M": M, "K": K, "dtype": dtype, "residual": residual, "out": out, "pad": pad}


def _norm_backward(name, M, K, dtype, residual, dw, accumulate, pad=0):
    return {"name": name, "op": "norm backward", "M": M, "K": K, "dtype": dtype, "residual": residual, "dw": dw,
            "accumulate": accumulate, "pad": pad}


def _linear_i8(name, M, N, K, dtype, act, bias, residual, save, pad=0):
    return {"name": name, "op": "linear i8", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "save": save, "pad": pad}


def _store(name, M, K, dtype, pad=0):
    return {"name": name, "op": "store", "M": M, "K": K, "dtype": dtype, "pad": pad}


def _backward(name, M, N, K, dtype, act, bias, z8, dw, accumulate, pad=0):
    return {"name": name, "op": "backward", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias, "z8": z8,
            "dw": dw, "accumulate": accumulate, "pad": pad}


def listed():
    return [
        # one token between two layers, as in serving: latency
        _norm("norm decode 1", 1, 8192, "bf16", True, "q8"),
        # a prompt whose rows are no multiple of a 16-byte vector, kept in 16 bits
        _norm("norm ragged 1000", 1000, 4100, "f16", True, "y", 3),
        # a long prompt or a training micro-batch, its output in 8 bits for the next layer and for the backward pass
        _norm("norm 16384", 16384, 8192, "bf16", True, "q8"),
        # gradients of a small norm: latency
        _norm_backward("norm backward 80", 80, 520, "f16", False, "f16", False),
        # gradients of a micro-batch's norm with the gradient from the residual's way, the weight's added up in 32 bits
        _norm_backward("norm backward 16384", 16384, 8192, "bf16", True, "f32", True),
        # one token through a layer with 8-bit weights: they are streamed once
        _linear_i8("i8 decode 1", 1, 3584, 8192, "bf16", "silu", True, False, False),
        # a short prompt
        _linear_i8("i8 prompt 1024", 1024, 3584, 8192, "bf16", "gelu", True, True, False),
        # a long prompt
        _linear_i8("i8 16384", 16384, 3584, 8192, "bf16", "none", False, True, False),
        # sizes that are no multiple of a tile or of a 16-byte vector, rows at odd addresses
        _linear_i8("i8 ragged 1000", 1000, 4100, 4100, "f16", "relu", True, False, True, 3),
        # a micro-batch's activations into 8 bits and back
        _store("store 16384", 16384, 8192, "bf16"),
        # gradients of a ragged layer whose input was kept in 8 bits
        _backward("backward ragged 1000", 1000, 4100, 4100, "f16", "relu", True, False, "f16", False),
        # gradients of a training micro-batch, input and pre-activation kept in 8 bits
        _backward("backward 16384", 16384, 3584, 8192, "bf16", "gelu_tanh", True, True, "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, n, least=64):
    """Half of the widths in whole vectors, as most models have them."""
    return max(least, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(("norm", "norm backward", "linear i8", "linear i8", "store", "backward", "backward"))
    dtype, pad = rng.choice(("bf16", "f16")), rng.choice((0, 0, 8, 3))
    if op in ("norm", "norm backward", "store"):
        K = _width(rng, _log(rng, 32, 32768))       # from the width of a head to that of the largest layers
        M = _log(rng, 1, min(131072, 16384 * 8192 // K))
        if op == "norm":
            return _unnamed(_norm("", M, K, dtype, rng.random() < 0.7, rng.choice(("y", "q8")), pad))
        if op == "store":
            return _unnamed(_store("", M, K, rng.choice((dtype, dtype, "f32")) if M * K <= 1 << 26 else dtype, pad))
        return _unnamed(_norm_backward("", M, K, dtype, rng.random() < 0.7, rng.choice((dtype, "f32")),
                                       rng.random() < 0.3, pad))
    M, N, K = _log(rng, 1, 16384), _width(rng, _log(rng, 64, 8192)), _width(rng, _log(rng, 64, 8192))
    while 2.0 * M * N * K > 2.0 * 16384 * 3584 * 8192:
        M = max(1, M // 2)
    act = rng.choice(ACTS)
    if op == "linear i8":
        return _unnamed(_linear_i8("", M, N, K, dtype, act, rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5, pad))
    return _unnamed(_backward("", M, N, K, dtype, act, rng.random() < 0.7, act != "none" and rng.random() < 0.5,
                              rng.choice((dtype, dtype, "f32")), rng.random() < 0.3, pad))


def _unnamed(case):
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _randn(gen, rows, cols, pad, dtype, scale=1.0):
    """A rows x cols matrix whose rows are cols + pad elements apart."""
    full = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32)
    return full.mul_(scale).to(dtype)[:, :cols]


def _activations(gen, rows, cols, pad, dtype):
    """Activations: rows of different size, and some channels far above the others."""
    full = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32)
    full *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    full *= torch.where(torch.rand(cols + pad, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    return full.to(dtype)[:, :cols]


def _empty(rows, cols, pad, dtype):
    return torch.empty(rows, cols + pad, device="cuda", dtype=dtype)[:, :cols]


def _codes_in(gen, rows, cols, pad, scale):
    """An 8-bit operand as a quantizer leaves it: bell-shaped codes, each row's largest 127, and the rows' scales."""
    v = torch.randn(rows, cols + pad, generator=gen, device="cuda")[:, :cols]
    top = v.abs().amax(1, keepdim=True)
    q = _empty(rows, cols, pad, torch.int8)
    q.copy_(torch.round(v * (127.0 / top)))
    return q, (top[:, 0] * (scale / 127.0)).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M, K, pad, dt = case["op"], case["M"], case["K"], case["pad"], TYPES[case["dtype"]]
    s = {"case": case}
    vector = lambda n, t: torch.empty(n, device="cuda", dtype=t)  # noqa: E731
    if op == "norm":
        s["x"] = _activations(gen, M, K, pad, dt)
        s["r"] = _activations(gen, M, K, pad, dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(dt)
        s["h"] = _empty(M, K, pad, dt) if case["residual"] else None
        if case["out"] == "y":
            s["y"], s["rstd"] = _empty(M, K, pad, dt), vector(M, torch.float32)
        else:
            s["q"], s["scale"], s["values"] = _empty(M, K, pad, torch.int8), vector(M, torch.float32), _empty(M, K, pad, dt)
    elif op == "norm backward":
        s["h"] = _activations(gen, M, K, pad, dt)
        s["rstd"] = (1.0 / torch.sqrt(s["h"].double().square().mean(1) + EPS)).float()
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(dt)
        s["dy"] = _randn(gen, M, K, pad, dt)
        s["dh"] = _randn(gen, M, K, pad, dt) if case["residual"] else None
        s["dx"], s["dw"] = _empty(M, K, pad, dt), vector(K, TYPES[case["dw"]])
        if case["accumulate"]:      # what the micro-batches before this one added up
            s["dw"].copy_(torch.randn(K, generator=gen, device="cuda"))
    elif op == "linear i8":
        N = case["N"]
        s["x"], s["x_scale"] = _codes_in(gen, M, K, pad, 1.0)
        s["w"], s["w_scale"] = _codes_in(gen, N, K, pad, 1.0 / math.sqrt(K))
        s["b"] = _randn(gen, 1, N, 0, dt, 0.1)[0] if case["bias"] else None
        s["r"] = _randn(gen, M, N, pad, dt) if case["residual"] else None
        s["y"] = _empty(M, N, pad, dt)
        s["z"] = _empty(M, N, pad, dt) if case["save"] else None
    elif op == "store":
        s["x"] = _activations(gen, M, K, pad, dt)
        s["q"], s["scale"] = _empty(M, K, pad, torch.int8), vector(M, torch.float32)
        s["values"] = _empty(M, K, pad, dt)
    else:
        N = case["N"]
        s["x"] = _activations(gen, M, K, pad, dt)
        s["x8"], s["x_scale"] = _empty(M, K, pad, torch.int8), vector(M, torch.float32)
        s["w"] = _randn(gen, N, K, pad, dt, 1.0 / math.sqrt(K))
        s["dy"] = _randn(gen, M, N, pad, dt)
        s["z"] = _randn(gen, M, N, pad, dt) if case["act"] != "none" else None
        if case["z8"]:
            s["z8"], s["z_scale"] = _empty(M, N, pad, torch.int8), vector(M, torch.float32)
        s["dx"], s["dw"] = _empty(M, K, pad, dt), _empty(N, K, pad, TYPES[case["dw"]])
        s["db"] = vector(N, TYPES[case["dw"]]) if case["bias"] else None
        if case["accumulate"]:
            s["dw"].copy_(_randn(gen, N, K, pad, TYPES[case["dw"]]))
            if case["bias"]:
                s["db"].copy_(_randn(gen, 1, N, 0, TYPES[case["dw"]])[0])
    if own and op in ("norm backward", "linear i8", "backward"):
        from gemm_all_gather_amd import binding as ag
        plan = {"norm backward": ag.plan_rms_norm_backward, "linear i8": ag.plan_linear_i8,
                "backward": ag.plan_linear_backward_q8}[op]
        s["workspace"] = torch.empty(max(1, plan(**_arguments(s)).workspace_bytes), device="cuda", dtype=torch.uint8)
    return s


def _stride(t):
    return 0 if t is None else t.stride(0)


def _arguments(s):
    """The keyword arguments of the library's call."""
    c = s["case"]
    a = {"M": c["M"], "K": c["K"], "dtype": c["dtype"]}
    if c["op"] == "norm":
        a.update(x=s["x"], residual=s["r"], weight=s["weight"], h=s["h"], eps=EPS, ldx=_stride(s["x"]), ldr=_stride(s["r"]),
                 ldh=_stride(s["h"]))
        if c["out"] == "y":
            a.update(y=s["y"], ldy=_stride(s["y"]), rstd=s["rstd"])
        else:
            a.update(q=s["q"], ldq=_stride(s["q"]), scale=s["scale"])
    elif c["op"] == "norm backward":
        a.update(dy=s["dy"], h=s["h"], rstd=s["rstd"], weight=s["weight"], dh=s["dh"], dx=s["dx"], dw=s["dw"],
                 lddy=_stride(s["dy"]), ldh=_stride(s["h"]), lddh=_stride(s["dh"]), lddx=_stride(s["dx"]),
                 dw_dtype=c["dw"], accumulate=c["accumulate"])
    elif c["op"] == "linear i8":
        a.update(N=c["N"], act=c["act"], x=s["x"], w=s["w"], x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["b"],
                 residual=s["r"], y=s["y"], z=s["z"], ldx=_stride(s["x"]), ldw=_stride(s["w"]), ldr=_stride(s["r"]),
                 ldy=_stride(s["y"]), ldz=_stride(s["z"]))
    else:
        z = s["z8"] if c["z8"] else s["z"]
        a.update(N=c["N"], act=c["act"], dy=s["dy"], x=s["x8"], x_scale=s["x_scale"], w=s["w"], z=z,
                 z_scale=s["z_scale"] if c["z8"] else None, dx=s["dx"], dw=s["dw"], db=s["db"], lddy=_stride(s["dy"]),
                 ldx=_stride(s["x8"]), ldw=_stride(s["w"]), ldz=_stride(z), lddx=_stride(s["dx"]), lddw=_stride(s["dw"]),
                 dw_dtype=c["dw"], accumulate=c["accumulate"])
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


def _codes(v):
    """Each row's codes, decided in 64 bits (ties to even), and its largest magnitude."""
    top = v.abs().amax(1, keepdim=True).double()
    return torch.round(v.double() * 127.0 / torch.where(top > 0, top, 1.0)).float(), top


def _plain_norm(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    h = (s["x"].float() + s["r"].float()).to(dt) if c["residual"] else s["x"]
    hf, w = h.float(), s["weight"].float()
    rstd = 1.0 / torch.sqrt((hf * hf).mean(1) + EPS)
    if c["out"] == "y":
        out = [(hf * rstd[:, None] * w).to(dt), rstd]
    else:
        codes, top = _codes(hf * w)                 # the product of two 16-bit numbers is exact in 32 bits
        scale = (top[:, 0] * rstd.double() / 127.0).float()
        out = [(codes * scale[:, None]).to(dt), scale]
    return ([h] if c["residual"] else []) + out


def _plain_norm_backward(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    dy, h, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    n = h * r
    g = dy * s["weight"].float()
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    if c["residual"]:
        dx = dx + s["dh"].float()
    dw = (dy * n).double().sum(0)
    if c["accumulate"]:
        dw = dw + s["dw"].double()
    s["dw"].copy_(dw)
    return [dx.to(dt), s["dw"]]


def _plain_linear_i8(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    z = (s["x"].float() @ s["w"].float().t()) * s["x_scale"][:, None] * s["w_scale"]
    if c["bias"]:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["r"].float()
    return [y.to(dt)] + ([z.to(dt)] if c["save"] else [])


def _kept(x):
    """What is left of x after 8 bits, in 32."""
    codes, top = _codes(x.float())
    return codes * (top / 127.0).float()


def _plain_store(s):
    scale = (s["x"].abs().amax(1).double() / 127.0).float()
    return [_kept(s["x"]).to(TYPES[s["case"]["dtype"]]), scale]


def _plain_backward(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(_kept(s["z"]) if c["z8"] else s["z"].float(), c["act"])
    dx = dz @ s["w"].float()
    dw = dz.t() @ _kept(s["x"])
    db = dz.double().sum(0).float() if c["bias"] else None
    if c["accumulate"]:
        dw = dw + s["dw"].float()
        db = db + s["db"].float() if c["bias"] else None
    s["dw"].copy_(dw)
    if c["bias"]:
        s["db"].copy_(db)
    return [dx.to(dt), s["dw"]] + ([s["db"]] if c["bias"] else [])


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"norm": _plain_norm, "norm backward": _plain_norm_backward, "linear i8": _plain_linear_i8,
                "store": _plain_store, "backward": _plain_backward}[op](s)
    from gemm_all_gather_amd import binding as ag
    stream = torch.cuda.current_stream()
    if op == "norm":
        ag.rms_norm(**_arguments(s), stream=stream)
        h = [s["h"]] if c["residual"] else []
        if c["out"] == "y":
            return h + [s["y"], s["rstd"]]
        # the values that the codes stand for
        ag.dequantize_rows(s["q"], s["scale"], s["values"], c["M"], c["K"], c["dtype"], ldq=_stride(s["q"]),
                           ldy=_stride(s["values"]), stream=stream)
        return h + [s["values"], s["scale"]]
    if op == "norm backward":
        ag.rms_norm_backward(**_arguments(s), workspace=s["workspace"], stream=stream)
        return [s["dx"], s["dw"]]
    if op == "linear i8":
        ag.linear_i8(**_arguments(s), workspace=s["workspace"], stream=stream)
        return [t for t in (s["y"], s["z"]) if t is not None]
    if op == "store":
        ag.quantize_rows(s["x"], s["q"], s["scale"], c["M"], c["K"], c["dtype"], ldx=_stride(s["x"]), ldq=_stride(s["q"]),
                         stream=stream)
        ag.dequantize_rows(s["q"], s["scale"], s["values"], c["M"], c["K"], c["dtype"], ldq=_stride(s["q"]),
                           ldy=_stride(s["values"]), stream=stream)
        return [s["values"], s["scale"]]
    # the forward pass keeps the activations in 8 bits, the backward pass reads them
    ag.quantize_rows(s["x"], s["x8"], s["x_scale"], c["M"], c["K"], c["dtype"], ldx=_stride(s["x"]), ldq=_stride(s["x8"]),
                     stream=stream)
    if c["z8"]:
        ag.quantize_rows(s["z"], s["z8"], s["z_scale"], c["M"], c["N"], c["dtype"], ldx=_stride(s["z"]), ldq=_stride(s["z8"]),
                         stream=stream)
    ag.linear_backward_q8(**_arguments(s), workspace=s["workspace"], stream=stream)
    return [t for t in (s["dx"], s["dw"], s["db"]) if t is not None]


# ------------------------------------------------------------------ the definition in 64 bits

def _quantized(v):
    """v as its row's codes stand for it, and the row's unit: the nearest whole number of units, an even one from between."""
    top = torch.amax(torch.abs(v), dim=1, keepdim=True)
    size, unit = torch.abs(v) * 127.0, torch.where(top > 0, top, 1.0)
    whole = torch.floor(size / unit)
    over = 2.0 * (size - whole * unit)
    up = (over > unit) | ((over == unit) & (torch.remainder(whole, 2.0) == 1.0))
    return torch.sign(v) * (whole + up) * top / 127.0, top[:, 0] / 127.0


def exact(case, seed):
    s = prepare(case, seed)
    f = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "norm":
        total = f(s["x"]) if s["r"] is None else f(s["x"]) + f(s["r"])
        h = f(s["x"] if s["r"] is None else total.to(TYPES[case["dtype"]]))      # the norm is of the rounded sum
        root = torch.rsqrt(torch.sum(h ** 2, dim=1) / case["K"] + EPS)
        out = [] if s["r"] is None else [total]
        if case["out"] == "y":
            return out + [h * torch.outer(root, f(s["weight"])), root]
        kept, unit = _quantized(h.mul_(f(s["weight"])))
        return out + [kept.mul_(root[:, None]), unit * root]
    if case["op"] == "norm backward":
        h, root, dy = f(s["h"]), f(s["rstd"]), f(s["dy"])
        g = dy * f(s["weight"])[None, :]
        along = torch.sum(g * h, dim=1) * root ** 3 / case["K"]
        dx = g.mul_(root[:, None]) - h * along[:, None]
        if s["dh"] is not None:
            dx += f(s["dh"])
        dw = torch.mv(dy.mul_(h).t(), root)
        return [dx, dw + f(s["dw"]) if case["accumulate"] else dw]
    if case["op"] == "store":
        return list(_quantized(f(s["x"])))
    if case["op"] == "linear i8":
        z = torch.matmul(f(s["x"]), f(s["w"]).transpose(0, 1).contiguous())
        z *= torch.outer(f(s["x_scale"]), f(s["w_scale"]))
        if s["b"] is not None:
            z += f(s["b"])[None, :]
        y = {"none": lambda: z, "relu": lambda: z.clamp(min=0.0), "gelu": lambda: z * torch.special.ndtr(z),
             "gelu_tanh": lambda: z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)),
             "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
        if s["r"] is not None:
            y = y + f(s["r"])
        return [y, z] if case["save"] else [y]
    dz = f(s["dy"])
    if case["act"] != "none":
        z = f(s["z"])
        if case["z8"]:
            z = _quantized(z)[0]
        sig = torch.sigmoid(z)
        u = 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
        du = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z ** 2)
        dz *= {"relu": lambda: (z > 0).double(),
               "gelu": lambda: torch.special.ndtr(z) + z * torch.exp(-z * z / 2.0) * (2.0 * math.pi) ** -0.5,
               "gelu_tanh": lambda: torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * du,
               "silu": lambda: sig + z * sig * (1.0 - sig)}[case["act"]]()
    out = [torch.matmul(dz, f(s["w"])), torch.matmul(dz.transpose(0, 1).contiguous(), _quantized(f(s["x"]))[0])]
    if case["bias"]:
        out.append(torch.sum(dz, dim=0))
    if case["accumulate"]:
        out[1] += f(s["dw"])
        if case["bias"]:
            out[2] += f(s["db"])
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    M, K = case["M"], case["K"]
    t = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        # codes, and the values that they stand for; or the rounded output
        each = t * (3 if case["residual"] else 1) + (t if case["out"] == "y" else 1 + t)
        return {"bytes": M * K * each + 4.0 * M + t * K, "flops": 5.0 * M * K}
    if case["op"] == "norm backward":
        d = 4 if case["dw"] == "f32" else 2
        return {"bytes": M * K * t * (4.0 if case["residual"] else 3.0) + 4.0 * M + t * K + d * K * (2 if case["accumulate"] else 1),
                "flops": 9.0 * M * K}
    if case["op"] == "store":
        return {"bytes": M * K * (2.0 * t + 1) + 4.0 * M, "flops": 3.0 * M * K}
    N = case["N"]
    if case["op"] == "linear i8":
        outs = 1 + case["residual"] + case["save"]
        return {"bytes": M * K + N * K + 4.0 * (M + N) + 2.0 * (outs * M * N + (N if case["bias"] else 0)), "flops": 2.0 * M * N * K}
    d = 4 if case["dw"] == "f32" else 2
    grads = (N * K + (N if case["bias"] else 0)) * (2 if case["accumulate"] else 1)
    reads = M * N * (2 if case["act"] != "none" else 1) + M * K + N * K
    kept = M * K + (M * N if case["z8"] else 0)
    return {"bytes": 2.0 * (reads + M * K) + kept + d * grads, "flops": 4.0 * M * N * K}
