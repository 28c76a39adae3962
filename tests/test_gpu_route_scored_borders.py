"""qw_route_scored where its choice is decided by little or by what is not a
number: ids, weights and grouping against the formula in 64 bits, as in
test_gpu_route_scored."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import tdt
from test_gpu_route_scored import logits, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E,n,top,k", [(24, 3, 1, 4), (24, 3, 2, 4), (256, 8, 4, 8), (256, 8, 1, 8), (1024, 8, 3, 8), (64, 32, 9, 9)])
def test_bias_of_nan(score, dtype, E, n, top, k):
    """An expert whose choice is NaN is not taken, and its group is valued by the
    others: NaN at the first, a middle and the last expert of groups, before
    and behind the largest, and in a whole group."""
    rng = np.random.default_rng(E + n)
    size = E // n
    for at in (0, 1, size // 2, size - 1):
        bias = (0.2 * rng.standard_normal(E)).astype(np.float32)
        bias[at::2 * size] = np.nan  # of every other group
        for by in ("max", "top2"):
            run(logits(67, E, at + 1), dtype, k, score, bias, n, top, by)
    bias[: (n - top) * size] = np.nan
    bias[(n - top) * size + size // 2] = np.inf
    run(logits(9, E, 70), dtype, k, score, bias, n, top, "top2")


@pytest.mark.parametrize("size", [1.0, 100.0, 1e3, 1e5])
@pytest.mark.parametrize("by", ["max", "top2"])
def test_biases_that_cancel(size, by):
    """Groups of two whose biases add up to nothing: a group's value is a small sum
    of large numbers."""
    rng = np.random.default_rng(int(size))
    bias = (size * rng.uniform(0.5, 1, (8, 1)) * [1, -1]).astype(np.float32).reshape(-1)
    run(logits(4000, 16, 71), "f32", 4, "sigmoid", bias, 8, 4, by)
    run(logits(4000, 16, 72), "f32", 4, "softmax", bias, 8, 4, by)


def test_a_large_bias_in_one_group():
    """One expert kept out by -1e9, one in by 1e6: the other groups' order is
    theirs."""
    bias = (0.1 * np.random.default_rng(8).standard_normal(64)).astype(np.float32)
    bias[3], bias[17] = -1e9, 1e6
    for n, top in ((8, 3), (32, 9), (1, 1)):
        for score in ("sigmoid", "softmax"):
            run(logits(3000, 64, 73), "f32", 6, score, bias, n, top, "top2")


# logits whose 64-bit scores are one number (1 above 37.5, 0 below -745 or that
# far below the largest, 1/2 next to 0), beside others
SAME = {"sigmoid": [38, 40, 45, 100, 3e4], "softmax": [-1e4, -1.5e4, -2e4, -3e4]}
LOW = [-768, -800, -896, -6e4]
TINY = [1e-30, 0.0, -1e-25, 3e-28, 1e-38]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,top", [(1, 1), (8, 3)])
@pytest.mark.parametrize("by", ["max", "top2"])
def test_a_token_does_not_depend_on_its_neighbours(score, dtype, n, top, by):
    """Tokens with scores that are equal in 64 bits though the logits are not, in
    every order, beside tokens that tie and ordinary ones: the formula's choice,
    and alone the same as among others."""
    import torch
    rng = np.random.default_rng(9)
    E, k, T = 64, 6, 96
    x = logits(T, E, 74)
    x[1::4] = np.round(x[1::4])  # ties
    for t in range(0, T, 4):
        if t % 8 == 0:
            x[t] = rng.choice(SAME[score] + ([] if t % 16 else [5.0]), E)
        else:
            x[t] = rng.choice(TINY + ([0.0] if t % 16 == 4 else [-3.0]), E)
        x[t + 2] = rng.choice(LOW if score == "sigmoid" else LOW + [0.0], E)
        x[t + 3, rng.choice(E, 10)] = rng.choice(SAME[score], 10)
    r = run(x, dtype, k, score, None, n, top, by)
    X = to_dev(x.astype(np.float32)).to(tdt(dtype))
    for t in range(T):
        one = qw.qw_route_scored(X[t:t + 1].contiguous(), k, score=score, n_groups=n, top_groups=top, group_by=by)
        assert torch.equal(one.ids[0], r.ids[t]) and torch.equal(one.weights[0], r.weights[t]), t
