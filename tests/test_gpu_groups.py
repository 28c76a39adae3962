"""GPU: grouping rows by id and the router's top-k, against the host's stable
sort and a 64-bit softmax. Ids, offsets and rows have to be equal; weights
are within a few fp32 roundings."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import F32, group, tdt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 511, 513, 2047, 2048, 2049, 5000, 70001])
@pytest.mark.parametrize("G", [1, 2, 8, 63, 64, 65, 300, 511, 512, 513, 1024])
def test_group_rows(n, G):
    rng = np.random.default_rng(n * 2000 + G)
    ids = rng.integers(-1, G + 1, n).astype(np.int32)  # -1 and G: no group
    off, rows = group(ids, G)
    g = qw.qw_group_rows(to_dev(ids), G)
    np.testing.assert_array_equal(g.offsets.cpu().numpy(), off)
    np.testing.assert_array_equal(g.rows.cpu().numpy(), rows)


@pytest.mark.parametrize("kind", ["none", "one", "last", "sorted", "extreme"])
@pytest.mark.parametrize("n", [100, 3000])
def test_group_rows_uneven(kind, n):
    G = 17
    ids = {"none": np.full(n, -1), "one": np.zeros(n), "last": np.full(n, G - 1), "sorted": np.arange(n) * G // n,
           "extreme": np.where(np.arange(n) % 3 == 0, -2**31, np.where(np.arange(n) % 3 == 1, 2**31 - 1, 5))}[kind]
    ids = ids.astype(np.int32)
    off, rows = group(ids, G)
    g = qw.qw_group_rows(to_dev(ids), G)
    np.testing.assert_array_equal(g.offsets.cpu().numpy(), off)
    np.testing.assert_array_equal(g.rows.cpu().numpy(), rows)


def route_ref(x, k, normalize):
    """ids, weights in 64 bits: largest first, ties to the lower index, NaN as -inf."""
    x = np.where(np.isnan(x), -np.inf, x)
    ids = np.argsort(-x, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(x, ids, 1)
    mx = np.where(np.isfinite(x.max(1, keepdims=True)), x.max(1, keepdims=True), 0.0)
    e = np.exp(x - mx)
    w = np.exp(top - mx)
    total = (w if normalize else e).sum(1, keepdims=True)
    w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return np.where(top > -np.inf, ids, -1).astype(np.int32), w


def check_route(x, k, normalize):
    import torch
    T, E = x.shape
    r = qw.qw_route_topk(x, k, normalize=normalize)
    ids, w = route_ref(x.double().cpu().numpy(), k, normalize)
    np.testing.assert_array_equal(r.ids.cpu().numpy(), ids)
    # exp's argument is one rounding off |l - max| at most, exp and the quotient a few steps, the sum E
    span = float(torch.nan_to_num(x.double(), 0, 0, 0).abs().max()) * 2
    tol = (span + E + 8) * F32 * w + 1e-37
    assert (np.abs(r.weights.double().cpu().numpy() - w) <= tol).all()
    off, rows = group(ids, E)
    np.testing.assert_array_equal(r.groups.offsets.cpu().numpy(), off)
    np.testing.assert_array_equal(r.groups.rows.cpu().numpy(), rows)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 2, 1), (17, 8, 2), (48, 64, 8), (5, 33, 9), (260, 60, 4),
                                   (257, 128, 8), (1000, 100, 6), (65, 129, 17), (40, 512, 32), (33, 1000, 10),
                                   (700, 1024, 32), (4097, 16, 1), (2049, 256, 3)])
def test_route(T, E, k, normalize, dtype):
    import torch
    torch.manual_seed(T + E + k)
    check_route((torch.randn(T, E, device="cuda") * 2).to(tdt(dtype)), k, normalize)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_ties_masks_and_nan(dtype, normalize):
    """Equal logits (both zeros among them), rows with few or no allowed
    experts, NaN, the types' lowest values, and large magnitudes."""
    import torch
    dt = tdt(dtype)
    torch.manual_seed(5)
    x = torch.randint(-2, 3, (300, 24), device="cuda").to(dt)
    x[::7] = 0.0
    x[::7, ::2] = -0.0
    x[1::7] = -torch.inf
    x[2::7, 3:] = -torch.inf
    x[3::7, ::3] = torch.nan
    x[4::7] = torch.finfo(dt).min
    x[5::7, 1] = 60000.0
    check_route(x, 6, normalize)


def test_route_is_the_same_each_time():
    import torch
    x = torch.randn(5000, 64, device="cuda")
    a = qw.qw_route_topk(x, 4)
    for _ in range(3):
        b = qw.qw_route_topk(x, 4)
        for s, t in ((a.ids, b.ids), (a.weights, b.weights), (a.groups.offsets, b.groups.offsets),
                     (a.groups.rows, b.groups.rows)):
            assert torch.equal(s, t)
