"""Shared helpers for the tests of the calls around a projection (not a test
module): one packed matrix with its 64-bit weights, and the products' formula
with its error bound."""

import math

import numpy as np

from routed_util import F32, Experts, half_step, tdt

TOP = {"e4m3": 448.0, "i8": 127.0}


def xdt(name):
    import torch
    return {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}.get(name) or tdt(name)


class Matrix(Experts):
    """A random packed matrix: pw, its weights W (N, K) in 64 bits and the
    magnitudes mag of the terms they are made of."""

    def __init__(self, fmt, N, K, n_out=0, seed=0):
        super().__init__(fmt, 1, N, K, n_out, seed)
        self.pw, self.W1, self.mag1 = self.packed[0], self.W[0], self.mag[0]


def activations(M, K, kind, seed):
    """(X, x_scales or None) on the device and their values in 64 bits, some
    channels larger than the others."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x[:, torch.randperm(K, generator=g)[: max(1, K // 50)]] *= 8
    if kind not in TOP:
        X = x.to(xdt(kind))
        return X.cuda(), None, X.double().numpy()
    s = x.abs().amax(1) / TOP[kind]
    q = x / s[:, None]
    X = (q.round() if kind == "i8" else q).to(xdt(kind))
    return X.cuda(), s.cuda(), X.double().numpy() * s.double().numpy()[:, None]


def act64(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * np.vectorize(math.erfc)(-z / math.sqrt(2)) if z.size else z
    if act == "gelu_tanh":
        return z / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def linear64(m, x64, kind, rounded, bias=None, act=None, gated=False, residual=None):
    """(values, bounds) of qgemm_linear in 64 bits; rounded: by the kernels
    that round the weights to 16 bits. All of the activations' slopes lie
    within -0.13 .. 1.13; an exponential, a quotient and the sums behind the
    product add a few fp32 roundings each."""
    import torch
    dt = torch.bfloat16 if kind == "bf16" else torch.float16  # of the operands
    extra = half_step(dt) ** 2 if m.fmt == "nf4" else 0.0  # a level is two numbers of dt
    small = 0.0
    if rounded and gated and kind == "bf16":
        # fp16 operands: what lies below 2^-28 of a row's largest is off by at most
        # 2^-39 of it (half of fp16's smallest step, 2^-25, where the largest is 2^14)
        dt = torch.float16
        small = 2.0 ** -39 * np.abs(x64).max(1, keepdims=True) * np.abs(m.W1).sum(1)[None]
    if rounded:
        extra = half_step(dt) + 2 * F32
    z = x64 @ m.W1.T
    tz = ((m.K + 64) * F32 + extra) * (np.abs(x64) @ m.mag1.T) + 2 * F32 * np.abs(z) + small
    if bias is not None:
        z = z + bias
        tz = tz + 2 * F32 * np.abs(z)
    if gated:
        g, u = np.split(z, 2, 1)
        tg, tu = np.split(tz, 2, 1)
        a = act64(g, act)
        ta = 1.13 * tg + 16 * F32 * np.abs(a)
        v = a * u
        tv = ta * (np.abs(u) + tu) + np.abs(a) * tu + F32 * np.abs(v)
    else:
        v = act64(z, act)
        tv = 1.13 * tz + 16 * F32 * np.abs(v)
    if residual is not None:
        v = v + residual
        tv = tv + F32 * (np.abs(v) + tv)
    return v, tv
