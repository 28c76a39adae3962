"""GPU: the router's weights, each within a bound of its own row: exp's
argument l - max is one rounding off, exp and the quotient a few steps, the
sum one rounding per expert."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from routed_util import F32, tdt

pytestmark = pytest.mark.gpu

GONE = 104.0  # exp(-104) is below every fp32 number
LEAST = 2.0**-126  # below fp32's normal numbers a weight may be flushed


def check(x, k, normalize):
    T, E = x.shape
    r = qw.qw_route_topk(x, k, normalize=normalize)
    l = x.double().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(l, ids, 1)
    mx = l.max(1, keepdims=True)
    mx = np.where(np.isfinite(mx), mx, 0.0)
    w, e = np.exp(top - mx), np.exp(l - mx)
    total = (w if normalize else e).sum(1, keepdims=True)
    want = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    np.testing.assert_array_equal(r.ids.cpu().numpy(), np.where(top > -np.inf, ids, -1))
    # the sum's own terms are off by |l - max| exp(l - max) <= 1 / e roundings each
    near = np.where(np.isfinite(top), np.minimum(np.abs(top - mx), GONE), 0.0)
    rel = (near + 2 * E + 16) * F32
    assert rel.max() < 2e-4
    got = r.weights.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= rel * want + LEAST)
    assert not bad.any(), f"{bad.sum()} of {bad.size}: {got[bad][:4]} for {want[bad][:4]}"
    assert (got[top == -np.inf] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
def test_ties_masks_nan_and_lowest_values(dtype, normalize):
    import torch
    dt = tdt(dtype)
    torch.manual_seed(7)
    for E, k in ((8, 8), (24, 6), (100, 7), (300, 20), (1000, 32)):
        x = torch.randint(-2, 3, (300, E), device="cuda").to(dt)
        x[::7] = 0.0
        x[::7, ::2] = -0.0
        x[1::7] = -torch.inf
        x[2::7, 3:] = -torch.inf
        x[3::7, ::3] = torch.nan
        x[4::7] = torch.finfo(dt).min
        x[4::14, 1] = torch.finfo(dt).max
        x[5::7, 1] = 60000.0
        check(x, k, normalize)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (48, 64, 8), (260, 60, 4), (1000, 256, 32), (4097, 128, 8), (70, 1024, 32)])
def test_spread_logits(T, E, k, normalize, dtype):
    """Logits apart by little and by much: some weights vanish."""
    import torch
    torch.manual_seed(T + E)
    for size in (0.01, 1.0, 30.0):
        check((torch.randn(T, E, device="cuda") * size).to(tdt(dtype)), k, normalize)
