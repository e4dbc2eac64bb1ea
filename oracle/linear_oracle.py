"""Linear layer, its gradients and the AdamW step in float64, from their definitions.

numpy only; shares no code with the library.  Matrices are float64 arrays of
the values that the 16-bit operands hold.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 256     # elements of an 8-bit state block

_erf = np.vectorize(math.erf, otypes=[np.float64])


def _sigmoid(u):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-u))


def act_oracle(z, act):
    if act == "none":
        return z
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * _sigmoid(z)
    raise ValueError(act)


def slope_oracle(z, act):
    """The derivative of act_oracle (relu: 0 at z <= 0)."""
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return np.where(z <= 0, 0.0, 1.0)
    if act == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        s = _sigmoid(z)
        return s + z * s * (1.0 - s)
    raise ValueError(act)


def linear_oracle(x, w, bias=None, act="none", residual=None):
    """(y, z): z = x w^T + bias, y = act(z) + residual."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = act_oracle(z, act)
    return (y if residual is None else y + residual), z


def linear_backward_oracle(dy, z, x, w, act="none"):
    """(dx, dw, db, dz) for the gradient dy of y."""
    dz = dy * slope_oracle(z, act) if act != "none" else dy
    return dz @ w, dz.T @ x, dz.sum(0), dz


# ------------------------------------------------------------------ AdamW

def random_bits_oracle(seed, place):
    """32 random bits of the state elements at the given places (counted in whole blocks over the tensors)."""
    whole = (1 << 64) - 1
    z = (seed + 0x9E3779B97F4A7C15) & whole         # the seed, spread over its 64 bits
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & whole
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & whole
    z ^= z >> 31
    m = np.uint64(0xFFFFFFFF)
    i = np.asarray(place, dtype=np.uint64)
    x = (i & m) ^ ((np.uint64(z & 0xFFFFFFFF) + (i >> np.uint64(32)) * np.uint64(0x9E3779B1)) & m)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x7FEB352D)) & m
    x = (x ^ (x >> np.uint64(15))) ^ np.uint64(z >> 32)
    x = (x * np.uint64(0x846CA68B)) & m
    return x ^ (x >> np.uint64(16))


def encode_oracle(value, power, top, u):
    """(codes, maxima) of non-negative values: value = (code/top)^power * maximum of its block of BLOCK."""
    n = value.size
    blocks = -(-n // BLOCK)
    v = np.zeros(blocks * BLOCK)
    v[:n] = value
    v = v.reshape(blocks, BLOCK)
    uu = np.full(blocks * BLOCK, 0.5)
    uu[:n] = u
    s = v.max(1).astype(np.float32)
    sd = s.astype(np.float64)[:, None]
    t = top * (v / np.where(sd > 0, sd, 1.0)) ** (1.0 / power)
    c = np.where(sd > 0, np.minimum(np.floor(t + uu.reshape(blocks, BLOCK)), top), 0.0)
    return c.reshape(-1)[:n], s


def decode_oracle(codes, maxima, power, top):
    """The values that codes stand for: |code|^power (a whole number) times maximum * (1 / top^power).

    The order of the operations is the definition's: a block's new maximum often lies exactly between two
    float32 numbers, and its side is then the last rounding's.
    """
    n = codes.size
    c = codes.astype(np.float64)
    scale = np.repeat(maxima.astype(np.float64), BLOCK)[:n] * (1.0 / top ** power)
    return np.sign(c) * np.abs(c) ** power * scale


def adamw_oracle(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after one step, all float64."""
    g = g * grad_scale
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + ((1.0 - beta2) * g) * g
    p = p * (1.0 - lr * weight_decay) - lr * (m / (1.0 - beta1 ** step)) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps)
    return p, m, v


def adamw8_codes_oracle(m, v, first_block, seed=None):
    """(m codes, m maxima, v codes, v maxima) of one tensor's new moments; seed None rounds to nearest."""
    n = m.size
    if seed is None:
        um = uv = np.full(n, 0.5)
    else:
        bits = random_bits_oracle(seed, np.arange(n, dtype=np.uint64) + np.uint64(first_block * BLOCK))
        um = (2.0 * (bits & np.uint64(0xFFFF)).astype(np.float64) + 1.0) / 131072.0
        uv = (2.0 * (bits >> np.uint64(16)).astype(np.float64) + 1.0) / 131072.0
    cm, ms = encode_oracle(np.abs(m), 2, 127.0, um)
    cv, vs = encode_oracle(v, 4, 255.0, uv)
    return cm * np.sign(m), ms, np.where(v > 0, np.maximum(cv, 1.0), cv), vs
