"""qw_route_scored against the formula in 64 bits: ids and grouping are equal,
weights off by their one rounding to fp32 and some 64-bit ones."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import F32, group, tdt

pytestmark = pytest.mark.gpu


def oracle(x, k, score, bias, n, top, by, normalize, scale):
    """(ids, weights) of logits x (T, E) in 64 bits."""
    T, E = x.shape
    here = x > -np.inf
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-x))
        else:
            e = np.where(here, np.exp(x - np.where(here, x, -1e300).max(1, keepdims=True)), 0.0)
            s = e / e.sum(1, keepdims=True)
        c = s + (0.0 if bias is None else bias.astype(np.float64))
    c = np.where(here & (c > -np.inf), c, -np.inf)
    if top < n:
        by_value = -np.sort(-c.reshape(T, n, E // n), axis=2)
        value = by_value[..., 0].copy()
        if by == "top2" and E // n > 1:
            value += np.where(by_value[..., 1] > -np.inf, by_value[..., 1], 0)
        order = np.argsort(-value, axis=1, kind="stable")
        keep = np.zeros((T, n), bool)
        np.put_along_axis(keep, order[:, :top], True, 1)
        c = np.where(np.repeat(keep, E // n, 1), c, -np.inf)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    taken = np.take_along_axis(c, ids, 1) > -np.inf
    w = np.where(taken, np.take_along_axis(s, ids, 1), 0.0)
    if normalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0.0)
    return np.where(taken, ids, -1).astype(np.int32), w * scale


def run(x, dtype, k, score="sigmoid", bias=None, n=1, top=None, by="top2", normalize=True, scale=1.0):
    X = to_dev(x.astype(np.float32)).to(tdt(dtype))
    top = n if top is None else top
    r = qw.qw_route_scored(X, k, score=score, bias=None if bias is None else to_dev(bias), n_groups=n, top_groups=top, group_by=by,
                           normalize=normalize, scale=scale)
    ids, w = oracle(X.double().cpu().numpy(), k, score, bias, n, top, by, normalize, scale)
    got = r.ids.cpu().numpy()
    assert np.array_equal(got, ids), (np.argwhere(got != ids)[:5], got[got != ids][:5], ids[got != ids][:5])
    gw = r.weights.double().cpu().numpy()
    assert (np.abs(gw - w) <= (F32 + 1e-12) * np.abs(w) + 2.0 ** -149).all()
    off, rows = group(ids, x.shape[1])
    assert np.array_equal(r.groups.offsets.cpu().numpy(), off) and np.array_equal(r.groups.rows.cpu().numpy(), rows)
    return r


def logits(T, E, seed):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((T, E)) * 2 + rng.standard_normal((1, E))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("by", ["max", "top2"])
@pytest.mark.parametrize("normalize", [False, True])
def test_forms(score, dtype, biased, by, normalize):
    bias = (0.1 * np.random.default_rng(1).standard_normal(64)).astype(np.float32) if biased else None
    run(logits(50, 64, 2), dtype, 6, score, bias, 8, 3, by, normalize, 2.5)


# (E, groups, top_groups, k): one group, groups of one expert, odd group sizes and
# numbers of groups, the most experts, groups and choices
@pytest.mark.parametrize("E,n,top,k", [(1, 1, 1, 1), (2, 2, 1, 1), (8, 8, 3, 3), (10, 5, 2, 4), (15, 3, 3, 7), (16, 1, 1, 16), (60, 4, 2, 5),
                                       (64, 64, 20, 20), (100, 5, 1, 20), (128, 4, 2, 32), (160, 8, 3, 6), (256, 8, 4, 8),
                                       (257, 1, 1, 8), (384, 6, 2, 8), (512, 32, 7, 9), (819, 63, 11, 32), (1024, 1, 1, 32),
                                       (1024, 64, 3, 32), (1023, 33, 5, 8), (1020, 17, 2, 4)])
@pytest.mark.parametrize("T", [1, 37])
def test_sizes(E, n, top, k, T):
    bias = (0.05 * np.random.default_rng(E).standard_normal(E)).astype(np.float32)
    run(logits(T, E, E + T), "f32", k, "sigmoid", bias, n, top, "top2", True, 1.0)


@pytest.mark.parametrize("T", [255, 2049, 20000])
def test_many_tokens(T):
    bias = (0.1 * np.random.default_rng(3).standard_normal(256)).astype(np.float32)
    run(logits(T, 256, T), "f32", 8, "sigmoid", bias, 8, 4, "top2", True, 2.5)


def test_ties_go_to_the_lower_expert_and_group():
    x = np.zeros((3, 32))
    r = run(x, "f32", 6, "sigmoid", None, 4, 2, "top2")
    assert r.ids.cpu().numpy().tolist() == [list(range(6))] * 3
    x[:, 20:24] = 1.0  # group 2 holds the largest, the other groups tie
    r = run(x, "bf16", 6, "softmax", None, 4, 2, "max")
    assert r.ids.cpu().numpy().tolist() == [[20, 21, 22, 23, 0, 1]] * 3
    # -0 and 0 are one value, and a bias may level what the logits do not
    x = np.where(np.arange(32) % 2, 0.0, -0.0)[None].repeat(2, 0)
    assert run(x, "f32", 4).ids.cpu().numpy().tolist() == [[0, 1, 2, 3]] * 2


def test_near_ties_are_told_apart_in_64_bits():
    """Logits so large that their fp32 sigmoids agree, next to each other in fp32."""
    top = np.float32(20.0)
    up = np.nextafter(top, np.float32(30))
    x = np.tile(np.array([top, up, top, np.nextafter(up, np.float32(30))], np.float32), (2, 4))
    r = run(x.astype(np.float64), "f32", 4)
    assert r.ids.cpu().numpy().tolist() == [[3, 7, 11, 15]] * 2
    # the bias makes up for all but the last bits of the scores' distance
    y = np.full((1, 4), -1.0)
    y[0, 2] = 0.5
    s = 1 / (1 + np.exp(-np.array([0.5, -1.0])))
    bias = np.array([0, np.float32(s[0] - s[1]), 0, 0], np.float32)
    run(y, "f32", 2, "sigmoid", bias)


def test_masked_experts_and_rows():
    """-inf and NaN logits, rows of nothing else, groups with one expert left or
    none, a bias of -inf, +inf logits."""
    x = logits(12, 24, 5)
    x[0] = -np.inf
    x[1, 1:] = -np.inf
    x[2, :8] = -np.inf
    x[3, 1:8] = np.nan
    x[4, ::2] = -np.inf
    x[5, 8:] = -np.inf
    x[6, 3] = np.inf
    bias = (0.2 * np.random.default_rng(6).standard_normal(24)).astype(np.float32)
    bias[9] = -np.inf
    for by in ("max", "top2"):
        for n, top in ((1, 1), (3, 2), (12, 5)):
            clean = np.where(np.isnan(x), -np.inf, x)
            a = run(clean, "f32", 4, "sigmoid", bias, n, top, by)
            b = qw.qw_route_scored(to_dev(x.astype(np.float32)), 4, bias=to_dev(bias), n_groups=n, top_groups=top, group_by=by)
            assert bool((a.ids == b.ids).all()) and bool((a.weights == b.weights).all())
            assert a.ids[0].tolist() == [-1] * 4 and a.weights[0].tolist() == [0] * 4
    x[6, 3] = 1.0
    run(np.where(np.isnan(x), -np.inf, x), "f32", 4, "softmax", bias, 3, 2, "top2")


def test_scores_that_underflow():
    """Sigmoids of -200 (1e-87) keep their order and their shares; of -800 they
    are zero, and so are the weights."""
    x = np.full((2, 8), -200.0) - np.arange(8) / 4
    run(x, "f32", 3)
    r = run(x * 4, "f32", 3)
    assert r.weights.cpu().numpy().tolist() == [[0.0] * 3] * 2


def test_without_bias_and_groups_it_is_the_softmax_router():
    """softmax scores without bias and groups choose what qw_route_topk chooses."""
    import torch
    X = to_dev(logits(300, 96, 7).astype(np.float32))
    for norm in (True, False):
        a = qw.qw_route_scored(X, 5, score="softmax", normalize=norm)
        b = qw.qw_route_topk(X, 5, normalize=norm)
        assert torch.equal(a.ids, b.ids) and torch.equal(a.groups.rows, b.groups.rows)
        assert torch.allclose(a.weights, b.weights, rtol=1e-5, atol=0)


def test_refusals_of_the_binding():
    import torch
    X = torch.zeros(4, 12, device="cuda")
    for kw in ({"score": "tanh"}, {"group_by": "sum"}, {"n_groups": 5}, {"n_groups": 4, "top_groups": 5}, {"n_groups": 6, "top_groups": 0},
               {"bias": torch.zeros(11, device="cuda")}):
        with pytest.raises(ValueError):
            qw.qw_route_scored(X, 2, **kw)
    with pytest.raises(ValueError):
        qw.qw_route_scored(X, 5, n_groups=3, top_groups=1)
    with pytest.raises(TypeError):
        qw.qw_route_scored(X, 2, bias=torch.zeros(12, device="cuda").half())
