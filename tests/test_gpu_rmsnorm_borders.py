"""qw_rmsnorm at the borders of the 8-bit grids and of its sizes.

Bound of an 8-bit element: a lane adds at most 32 squares in fp32 (each of a sum
rounded once: (32 + 2) 2^-24 of their sum at most, half of that in the root) and
everything behind that is in 64 bits but h's own rounding and three of the
element: less than 24 2^-24 of the element beside the half step of its grid."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from layer_util import TOP, xdt
from routed_util import F32
from test_gpu_rmsnorm import formula, inputs

pytestmark = pytest.mark.gpu


def nearest(n, want, kind, rel=24 * F32):
    """The elements of n are the nearest to want over their row's scale."""
    s = n.scales.double().cpu().numpy()
    v = n.y.double().cpu().numpy() if kind == "i8" else n.y.float().double().cpu().numpy()
    q = want / s[:, None]
    half = 0.5 if kind == "i8" else np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10)
    bad = ~(np.abs(v - q) <= half + rel * np.abs(q))
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], v[bad][:3], q[bad][:3])
    assert np.abs(v).max() <= TOP[kind]


@pytest.mark.parametrize("y", ["e4m3", "i8"])
@pytest.mark.parametrize("K", [1, 7, 64, 511, 520, 2048, 2056, 5120, 8191, 8192, 16384, 20001, 32768])
def test_permuted_8_bit_rows_are_the_plain_ones(K, y):
    """With perm, scales and elements are those without it, bit for bit, in the
    other order; entries out of range give zeros. Both are the nearest."""
    import torch
    M = 100
    X, R, W, P = inputs(M, K, "bf16", "f32", K + 1, "f32")
    plain = qw.qw_rmsnorm(X.cuda(), W.cuda(), residual=R.cuda(), out_dtype=xdt(y))
    bad = P.clone()
    if K > 8:
        bad[5], bad[6] = -1, K
    n = qw.qw_rmsnorm(X.cuda(), W.cuda(), residual=R.cuda(), perm=bad.cuda(), out_dtype=xdt(y))
    assert torch.equal(n.scales, plain.scales)
    want = plain.y.view(torch.uint8)[:, P.cuda().long()]
    if K > 8:
        want[:, 5:7] = 0
    got = n.y.view(torch.uint8)
    assert torch.equal(got, want), f"{int((got != want).sum())} of {got.numel()}"
    nearest(plain, formula(X, R, W, 1e-6)[1], y)


@pytest.mark.parametrize("perm", [False, True])
@pytest.mark.parametrize("y", ["e4m3", "i8"])
def test_8_bit_rows_of_tiny_numbers(y, perm):
    """eps = 0 and rows of 1e-10 by weights of 1e-27 (a row's factor is past fp32's
    largest number) and of zeros (the least scale, and zeros)."""
    import torch
    K = 640
    X, _, _, P = inputs(5, K, "f32", None, 11)
    X = X * 1e-10
    for w in (1e-27, 0.0):
        W = torch.full((K,), w)
        n = qw.qw_rmsnorm(X.cuda(), W.cuda(), 0.0, perm=P.cuda() if perm else None, out_dtype=xdt(y))
        want = formula(X, None, W, 0.0)[1]
        if w:
            nearest(n, want[:, P.numpy()] if perm else want, y)
        else:
            assert bool((n.scales == 2.0 ** -100).all()) and bool((n.y.view(torch.uint8) & 0x7F == 0).all())


def test_as_many_rows_as_a_call_takes():
    """2^24 rows of 513: 2^32 threads, more than one launch may have."""
    import torch
    M, K = qw.QW_MAX_ROWS, 513
    row = torch.randn(K, device="cuda").half()
    x = row.expand(M, K).contiguous()
    ends = torch.randn(2, 40, K, device="cuda").half()
    x[:40], x[-40:] = ends[0], ends[1]
    w = torch.randn(K, device="cuda").half()
    y = qw.qw_rmsnorm(x, w, out=x).y
    one = qw.qw_rmsnorm(row[None], w).y
    assert torch.equal(y[:40], qw.qw_rmsnorm(ends[0], w).y) and torch.equal(y[-40:], qw.qw_rmsnorm(ends[1], w).y)
    for at in range(40, M - 40, 1 << 20):
        assert torch.equal(y[at:at + 1], one), at
    at = (1 << 24) - (1 << 19)
    assert bool((y[at:-40] == one).all())


@pytest.mark.parametrize("y", ["e4m3", "i8"])
@pytest.mark.parametrize("x", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("K", [7, 512, 2048, 5120, 8192, 16384, 32768])
def test_scales_are_the_formulas_rounded_once(K, x, y):
    """A row's scale is off by half a step of fp32 and some 64-bit roundings, an element
    nearest to its number but for two roundings of it (the factor's and its own);
    rows of 1e25, whose squares fp32 cannot hold, too."""
    X, _, W, P = inputs(200, K, x, None, K + 2, "f32")
    if x != "f16":
        X[::50] = X[::50] * 1e25
    want = formula(X, None, W, 1e-6)[1]
    for perm in (None, P):
        n = qw.qw_rmsnorm(X.cuda(), W.cuda(), perm=None if perm is None else perm.cuda(), out_dtype=xdt(y))
        s = np.abs(want).max(1) / TOP[y]
        assert (np.abs(n.scales.double().cpu().numpy() - s) <= F32 * (1 + 2.0 ** -20) * s).all()
        nearest(n, want if perm is None else want[:, perm.numpy()], y, 2 * F32)
