"""qw_route_scored where its choice is decided by little or by what is not a
number: ids, weights and grouping against the formula in 64 bits, as in
test_gpu_route_scored."""

import numpy as np
import pytest

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
