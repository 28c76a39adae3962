"""Shared helpers for the tests of products whose rows take different
matrices (not a test module): packed experts with their 64-bit weights, row
groups, and the error bounds of the products.

A bound is what the arithmetic allows, elementwise: K (or r) fp32 additions
of products whose magnitudes sum to ``mag`` are off by at most K 2^-24 mag;
a value rounded to a type is off by at most half a step, eps / 2 of it.
"""

import numpy as np

import oracle
from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev

FMTS = {"2bit": qw.QW_FMT_2BIT_G32, "nf4": qw.QW_FMT_NF4_B64, "int4": qw.QW_FMT_INT4_G32}
F32 = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def tdt(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


class Experts:
    """E random experts packed by the library. W: the dequantized weights
    (E, N, K) in 64 bits, anchors in place; mag: the magnitudes of the terms
    each weight is made of (2-bit: |S C| + |Z|)."""

    def __init__(self, fmt, E, N, K, n_out=0, seed=0):
        rng = np.random.default_rng(seed)
        packed, W, mag = [], [], []
        for e in range(E):
            w = (rng.standard_normal((N, K)) * 0.02 * (1 + e % 3)).astype(np.float32)
            if fmt == "2bit":
                idx = np.sort(rng.choice(K, n_out, replace=False)).astype(np.int32) if n_out else None
                p = qw.qw_pack(to_dev(w), FMTS[fmt], to_dev(idx) if n_out else None)
                sz = p.host_scales().astype(np.float64)
                q = oracle.unpack_2bit(p.host_codes())
                d = oracle.dequant_2bit(q, sz[..., 0], sz[..., 1])
                m = np.abs(np.repeat(sz[..., 0], 32, 1) * oracle.CODEBOOK[q]) + np.abs(np.repeat(sz[..., 1], 32, 1))
            elif fmt == "nf4":
                idx, p = None, qw.qw_pack(to_dev(w), FMTS[fmt])
                d = oracle.dequant_nf4(oracle.unpack_nf4(p.host_codes()), p.host_scales().astype(np.float64))
                m = np.abs(d)
            else:
                idx = np.arange(n_out)
                p = qw.qw_pack_int4(to_dev(w), to_dev(np.arange(K, dtype=np.int32)), n_out)
                d = oracle.dequant_int4(oracle.unpack_int4(p.host_codes()), p.host_scales().astype(np.float64))
                m = np.abs(d)
            if n_out:
                d[:, idx] = p.host_out_w()[:, :n_out].astype(np.float64)
                m[:, idx] = np.abs(d[:, idx])
            packed.append(p)
            W.append(d)
            mag.append(m)
        self.fmt, self.E, self.N, self.K = fmt, E, N, K
        self.packed, self.W, self.mag = packed, np.stack(W), np.stack(mag)
        self.ew = qw.ExpertWeights.stack(packed)


def group(ids, G):
    """The grouping of ids on the host: offsets and rows, ungrouped rows last."""
    ids = np.asarray(ids).reshape(-1).astype(np.int64)
    key = np.where((ids < 0) | (ids >= G), G, ids)
    rows = np.argsort(key, kind="stable").astype(np.int32)
    count = np.bincount(key, minlength=G + 1)[:G]
    return np.concatenate([[0], np.cumsum(count)]).astype(np.int32), rows


def device_groups(ids, G):
    off, rows = group(ids, G)
    return qw.RowGroups(to_dev(off), to_dev(rows)), off, rows


def products(ex, x64, off, wide, dtype, tall=False):
    """(values, bounds) of the rows in grouped order: row p times its group's
    weights; wide, tall: by the kernels of wide and of tall tiles."""
    y = np.zeros((x64.shape[0], ex.N))
    tol = np.zeros_like(y)
    extra = 0.0
    if ex.fmt == "nf4":  # a level is two numbers of dtype, in wide tiles one
        extra = half_step(dtype) if wide else half_step(dtype) ** 2
    elif ex.fmt == "2bit" and wide:  # Z and the group sums of x as two bf16 numbers, without the product of the rests
        extra = 2.0 ** -15
    if tall:  # every weight is rounded to dtype (and to fp32 before)
        extra = half_step(dtype) + F32
    for e in range(ex.E):
        s = slice(off[e], off[e + 1])
        y[s] = x64[s] @ ex.W[e].T
        tol[s] = ((ex.K + 64) * F32 + extra) * (np.abs(x64[s]) @ ex.mag[e].T)
    return y, tol


def gated(y, tol):
    """silu(gate) * up and its bound: silu' lies within -0.1..1.1, and the
    exponential, the quotient and the products add a few fp32 roundings."""
    g, u = np.split(y, 2, 1)
    tg, tu = np.split(tol, 2, 1)
    silu = g / (1 + np.exp(-g))
    v = silu * u
    return v, 1.1 * tg * (np.abs(u) + tu) + np.abs(silu) * tu + 16 * F32 * np.abs(v)


def assert_close(got, want, tol, dtype, what=""):
    """|got - want| <= tol plus the one rounding to dtype (and its smallest
    step, for values below its normal range)."""
    import torch
    got = got.double().cpu().numpy()
    lim = tol + half_step(dtype) * (np.abs(want) + tol) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[:3].tolist()}: "
                           f"{got[bad][:3]} for {want[bad][:3]}, allowed {lim[bad][:3]}")
