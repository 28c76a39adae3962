"""qw_rmsnorm against the formula in 64 bits.

Bounds: the sum x + residual is rounded once to fp32 (relative 2^-24, so
2 2^-24 of its square); the K squares are added in fp32 in any order (K 2^-24 of
their sum at most); the quotient, the root, the division and the products add
less than 8 roundings: y is off by at most (K / 2 + 16) 2^-24 |y| before its own
rounding. An 8-bit element is the nearest to its number, so off by half a step
(int8: half; e4m3: 2^-4 of the number, at least 2^-10) plus that bound."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from layer_util import TOP, xdt
from routed_util import F32, assert_close, half_step, tdt

pytestmark = pytest.mark.gpu


def inputs(M, K, x, r, seed, w=None):
    import torch
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(M, K, generator=g).to(tdt(x))
    R = (4 * torch.randn(M, K, generator=g)).to(tdt(r)) if r else None
    W = (1 + 0.3 * torch.randn(K, generator=g)).to(tdt(w or x))
    return X, R, W, torch.randperm(K, generator=g).to(torch.int32)


def formula(X, R, W, eps):
    h = X.double() + (R.double() if R is not None else 0.0)
    return h.numpy(), (h / ((h * h).mean(1, keepdim=True) + eps).sqrt() * W.double()).numpy()


def check(n, h, y, kind, K):
    got = n.y
    rel = (K / 2 + 16) * F32
    if kind not in TOP:
        assert n.scales is None
        assert_close(got, y, rel * np.abs(y), got.dtype, "y")
        return
    largest = np.abs(y).max(1)
    s = n.scales.double().cpu().numpy()
    want = np.maximum(largest / TOP[kind], 2.0 ** -100)
    assert (np.abs(s - want) <= rel * want).all()
    v = got.double().cpu().numpy() if kind == "i8" else got.float().double().cpu().numpy()
    q = y / s[:, None]
    half = 0.5 if kind == "i8" else np.maximum(2.0 ** -4 * np.abs(q), 2.0 ** -10)
    assert (np.abs(v - q) <= half + 2 * rel * np.abs(q)).all()
    assert np.abs(v).max() <= TOP[kind]


@pytest.mark.parametrize("y", ["f16", "bf16", "f32", "e4m3", "i8"])
@pytest.mark.parametrize("x,r", [("f16", None), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_types(x, r, y):
    M, K = 5, 1024
    X, R, W, _ = inputs(M, K, x, r, 1)
    n = qw.qw_rmsnorm(X.cuda(), W.cuda(), 1e-5, residual=R.cuda() if r else None, out_dtype=xdt(y))
    h, want = formula(X, R, W, 1e-5)
    check(n, h, want, y, K)
    if r:
        assert_close(n.residual, h, F32 * np.abs(h), tdt(r), "residual")
    else:
        assert n.residual is None


@pytest.mark.parametrize("perm", [False, True])
@pytest.mark.parametrize("y", ["f16", "e4m3", "i8"])
@pytest.mark.parametrize("K", [1, 2, 7, 8, 63, 64, 511, 512, 520, 2048, 2056, 4095, 4096, 4104, 8191, 8192, 8200, 16384, 16392,
                               20001, 32768])
def test_widths(K, y, perm):
    M = 3
    X, R, W, P = inputs(M, K, "f16", "f16", K)
    n = qw.qw_rmsnorm(X.cuda(), W.cuda(), 1e-6, residual=R.cuda(), perm=P.cuda() if perm else None, out_dtype=xdt(y))
    h, want = formula(X, R, W, 1e-6)
    check(n, h, want[:, P.numpy()] if perm else want, y, K)
    assert_close(n.residual, h, F32 * np.abs(h), tdt("f16"), "residual")


@pytest.mark.parametrize("M", [1, 2, 4, 5, 63, 300, 5000])
@pytest.mark.parametrize("K", [96, 1000, 5120])
def test_rows(M, K):
    X, R, W, P = inputs(M, K, "bf16", "bf16", M, "f32")
    n = qw.qw_rmsnorm(X.cuda(), W.cuda(), 1e-6, residual=R.cuda(), out_dtype=tdt("f32"))
    h, want = formula(X, R, W, 1e-6)
    check(n, h, want, "f32", K)


def test_in_place_and_given_outputs():
    import torch
    M, K = 70, 5120
    X, R, W, P = inputs(M, K, "bf16", "bf16", 3)
    want = qw.qw_rmsnorm(X.cuda(), W.cuda(), residual=R.cuda(), perm=P.cuda())
    x, r = X.cuda(), R.cuda()
    n = qw.qw_rmsnorm(x, W.cuda(), residual=r, residual_out=r, perm=P.cuda(), out=x)
    assert n.y is x and n.residual is r
    assert torch.equal(x, want.y) and torch.equal(r, want.residual)
    ws, wy = torch.full((M,), 7.0, device="cuda"), torch.empty(M, K, dtype=torch.int8, device="cuda")
    n = qw.qw_rmsnorm(X.cuda(), W.cuda(), out=wy, scales=ws)
    assert n.y is wy and n.scales is ws and float(ws.max()) < 1


def test_permuted_rows_are_the_products_order():
    """perm leaves what qw_permute_cols of the plain norm leaves, bit for bit."""
    import torch
    X, R, W, P = inputs(9, 1536, "f16", "f32", 4)
    plain = qw.qw_rmsnorm(X.cuda(), W.cuda(), residual=R.cuda())
    n = qw.qw_rmsnorm(X.cuda(), W.cuda(), residual=R.cuda(), perm=P.cuda())
    assert torch.equal(n.y, qw.qw_permute_cols(plain.y, P.cuda()))
    bad = P.clone()
    bad[5], bad[6] = -1, 1536
    y = qw.qw_rmsnorm(X.cuda(), W.cuda(), residual=R.cuda(), perm=bad.cuda()).y
    assert bool((y[:, 5:7] == 0).all()) and torch.equal(y[:, 7:], n.y[:, 7:])


@pytest.mark.parametrize("y", ["f16", "e4m3", "i8"])
def test_rows_of_zeros_tiny_and_not_finite(y):
    """Row by row: zeros, tiny values, an infinity, a NaN, ordinary ones; no row
    touches another."""
    import torch
    K = 640
    X = torch.randn(5, K, generator=torch.Generator().manual_seed(5))
    X[0] = 0
    X[1] *= 1e-30
    X[2, 17], X[3, 600] = float("inf"), float("nan")
    W = torch.ones(K)
    n = qw.qw_rmsnorm(X.cuda(), W.cuda(), 1e-6, out_dtype=xdt(y))
    v = n.y.float().cpu() if y != "i8" else n.y.cpu().float()
    if n.scales is not None:
        s = n.scales.cpu()
        assert torch.isnan(s[2:4]).all() and torch.isfinite(s[[0, 1, 4]]).all() and float(s[0]) == 2.0 ** -100
        assert bool((v[2:4] == 0).all())
    else:
        assert torch.isnan(v[2, 17]) and torch.isnan(v[3]).all()
    assert bool((v[0] == 0).all())
    h, want = formula(X[[1, 4]], None, W, 1e-6)
    sub = qw.Normed(n.y[[1, 4]] if y == "i8" else n.y.view(torch.uint8)[[1, 4]].view(torch.float8_e4m3fn) if y == "e4m3" else n.y[[1, 4]],
                    None if n.scales is None else n.scales[[1, 4]], None)
    check(sub, h, want, y, K)


def test_refusals_of_the_binding():
    import torch
    X, R, W, P = (t.cuda() for t in inputs(4, 64, "f16", "f16", 6))
    for kw in ({"residual": R[:2]}, {"residual_out": R}, {"residual": R, "residual_out": R.float()}, {"perm": P[:32]},
               {"scales": torch.zeros(4, device="cuda")}, {"out": torch.empty(4, 65, device="cuda")},
               {"out": torch.empty(4, 64, dtype=torch.float64, device="cuda")}, {"residual": R.t().contiguous().t()},
               {"out_dtype": torch.int8, "scales": torch.zeros(5, device="cuda")}):
        with pytest.raises((ValueError, TypeError)):
            qw.qw_rmsnorm(X, W, **kw)
    with pytest.raises(ValueError):
        qw.qw_rmsnorm(X, W[:32])
    with pytest.raises(TypeError):
        qw.qw_rmsnorm(X.double(), W)
