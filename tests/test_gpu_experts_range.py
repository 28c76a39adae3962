"""GPU: the experts' products with fp16 activations over weights far from 1,
by every tile height. The tall tiles round each weight to fp16, whose normal
numbers end at 2^-14 and 65504; a weight beyond them has to come through with
the same relative error as one within. Bounds are those of routed_util."""

import numpy as np
import pytest

import oracle
from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import FMTS, F32, assert_close, device_groups, half_step

pytestmark = pytest.mark.gpu

GROUP = {"2bit": 32, "nf4": 64, "int4": 32}


def experts(fmt, E, N, K, scale, rng):
    """Experts of random codes and the given scales (E, N, K / group; 2-bit:
    with a tenth of it as offset), their weights and the magnitudes of the
    terms each is made of, in 64 bits."""
    if fmt == "2bit":
        q = rng.integers(0, 4, (E, N, K))
        codes = (q.reshape(E, N, -1, 4) << np.array([0, 2, 4, 6])).sum(-1).astype(np.uint8)
        sz = np.stack([scale, 0.1 * scale * rng.standard_normal(scale.shape)], -1).astype(np.float16)
        S, Z = (np.repeat(sz[..., i].astype(np.float64), 32, -1) for i in (0, 1))
        W = S * oracle.CODEBOOK[q] + Z
        mag = np.abs(S * oracle.CODEBOOK[q]) + np.abs(Z)
        scales = sz
    else:
        q = rng.integers(0, 16, (E, N, K)) if fmt == "nf4" else rng.integers(1, 16, (E, N, K))
        codes = (q.reshape(E, N, -1, 2) << np.array([0, 4])).sum(-1).astype(np.uint8)
        scales = scale.astype(np.float32 if fmt == "nf4" else np.float16)
        level = qw.qw_nf4_levels().astype(np.float64)[q] if fmt == "nf4" else q - 8.0
        W = level * np.repeat(scales.astype(np.float64), GROUP[fmt], -1)
        mag = np.abs(W)
    assert np.isfinite(W).all()
    return qw.ExpertWeights(FMTS[fmt], E, N, K, 0, to_dev(codes), to_dev(scales)), W, mag


def bound(fmt, K, blocks, x64, mag):
    """K fp32 additions, and the rounding of what enters the product: in tall
    tiles the weight (and its fp32 value before), in wide ones an NF4 level
    or the group sums against Z (two bf16 numbers each)."""
    import torch
    half = half_step(torch.float16)
    extra = half + F32 if blocks >= 8 else {"nf4": half if blocks > 1 else half**2,
                                            "2bit": 2.0**-15 if blocks > 1 else 0.0, "int4": 0.0}[fmt]
    return ((K + 64) * F32 + extra) * (np.abs(x64) @ mag.T)


def check(fmt, scale, blocks, x, rng):
    import torch
    E, N, K = scale.shape[0], scale.shape[1], scale.shape[2] * GROUP[fmt]
    ew, W, mag = experts(fmt, E, N, K, scale, rng)
    n = x.shape[0]
    g, off, rows = device_groups(rng.integers(0, E, n).astype(np.int32), E)
    Y = qw.qgemm_experts(ew, to_dev(x), g, out_dtype=torch.float32)
    x64 = x.astype(np.float64)[rows]
    want, tol = np.zeros((n, N)), np.zeros((n, N))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        want[s], tol[s] = x64[s] @ W[e].T, bound(fmt, K, blocks, x64[s], mag[e])
    assert_close(Y, want, tol, torch.float32, f"{fmt}, {blocks} blocks")


SIZES = [("2bit", s) for s in (2e-6, 1e-5, 1e-3, 40000.0)] + \
        [("int4", s) for s in (2e-6, 1e-5, 1e-3, 60000.0)] + \
        [("nf4", s) for s in (1e-30, 1e-8, 1e-6, 1e-5, 1e-4, 1e6, 1e30)]


@pytest.mark.parametrize("blocks", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("fmt,size", SIZES)
def test_small_and_large_weights(fmt, size, blocks, tune):
    """All weights of one size, small or large."""
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    rng = np.random.default_rng(1)
    for N, K in ((72, 64), (300, 448)):
        scale = size * rng.uniform(0.5, 1.0, (2, N, K // GROUP[fmt]))
        check(fmt, scale, blocks, rng.standard_normal((90, K)).astype(np.float16), rng)


@pytest.mark.parametrize("blocks", [1, 4, 8, 16])
@pytest.mark.parametrize("fmt,low", [("2bit", 2e-6), ("int4", 2e-6), ("nf4", 1e-12)])
def test_columns_of_different_sizes(fmt, low, blocks, tune):
    """Each column and expert with a size of its own, some of them zero: a
    column's result does not depend on its neighbours' sizes."""
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    rng = np.random.default_rng(2)
    N, K = 290, 320
    scale = np.exp(rng.uniform(np.log(low), np.log(2e4), (3, N, 1))) * rng.uniform(0.5, 1.0, (3, N, K // GROUP[fmt]))
    scale[:, ::17] = 0.0
    check(fmt, scale, blocks, rng.standard_normal((130, K)).astype(np.float16), rng)


@pytest.mark.parametrize("blocks", [1, 4, 8, 16])
@pytest.mark.parametrize("fmt", ["2bit", "int4", "nf4"])
def test_groups_of_different_sizes_seen_one_by_one(fmt, blocks, tune):
    """Groups of one column that differ by up to 2^20, against rows of X
    that are 1 in one channel: each weight is seen alone, to its own error."""
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    rng = np.random.default_rng(3)
    N, K = 70, 256
    scale = np.exp(rng.uniform(np.log(2e-5), np.log(20.0), (2, N, K // GROUP[fmt])))
    check(fmt, scale, blocks, np.eye(K, dtype=np.float16), rng)


@pytest.mark.parametrize("fmt,size", [("nf4", 1e-6), ("nf4", 1e6), ("int4", 1e-5), ("2bit", 40000.0)])
def test_automatic_choice_with_few_and_many_rows(fmt, size):
    """The same weights by a small and a large batch."""
    rng = np.random.default_rng(4)
    scale = size * rng.uniform(0.5, 1.0, (2, 512, 512 // GROUP[fmt]))
    for n in (3, 1000):
        check(fmt, scale, 8 if n > 3 else 1, rng.standard_normal((n, 512)).astype(np.float16), rng)


@pytest.mark.parametrize("blocks", [8, 16])
def test_scales_that_are_not_finite_stay_in_their_columns(blocks, tune):
    import torch
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    rng = np.random.default_rng(5)
    N, K = 96, 256
    for fmt in ("2bit", "int4", "nf4"):
        ew, _, _ = experts(fmt, 1, N, K, rng.uniform(0.01, 0.02, (1, N, K // GROUP[fmt])), rng)
        x = to_dev(rng.standard_normal((40, K)).astype(np.float16))
        g, *_ = device_groups(np.zeros(40), 1)
        clean = qw.qgemm_experts(ew, x, g, out_dtype=torch.float32)
        s = ew.scales.view(1, N, -1)
        s[0, 3, 1], s[0, 40, 0] = torch.inf, torch.nan
        Y = qw.qgemm_experts(ew, x, g, out_dtype=torch.float32)
        keep = torch.ones(N, dtype=torch.bool, device="cuda")
        keep[[3, 40]] = False
        assert torch.equal(Y[:, keep], clean[:, keep])
        assert not bool(torch.isfinite(Y[:, ~keep]).any())
