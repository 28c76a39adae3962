"""CPU checks of qgemm_linear's choice of kernel, by the workspace that it asks
for: parts of K (fp32 sums) are what tall tiles take, narrow ones take none."""

import ctypes
import os

import pytest

from bit_weight_quantized_qw_amd import qw

P = 0x1000  # stands for a device address
FMTS = {"2bit": qw.QW_FMT_2BIT_G32, "nf4": qw.QW_FMT_NF4_B64, "int4": qw.QW_FMT_INT4_G32}


@pytest.fixture(scope="module")
def size():
    if not os.path.exists(qw.LIB_PATH):
        from bit_weight_quantized_qw_amd.build import build
        build()

    def size(fmt, anchors, M, N, K, dtype=qw.QW_DT_BF16):
        pad = (anchors + 7) // 8 * 8
        a = P if anchors else None
        w = qw.qw_weight(FMTS[fmt], N, K, anchors, pad, P, P, a, a, a)
        return qw.lib().qw_linear_workspace_bytes(ctypes.byref(w), dtype, M, 0)
    return size


@pytest.mark.parametrize("fmt,anchors", [("2bit", 0), ("2bit", 300), ("int4", 82)])
@pytest.mark.parametrize("M", [33, 40, 64, 100])
@pytest.mark.parametrize("N", [16, 500, 1024])
def test_few_columns_and_long_sums_take_parts_of_K(size, fmt, anchors, M, N):
    """A narrow grid would leave most CUs empty, each of the others with all of K."""
    for K in (8192, 28672):
        assert size(fmt, anchors, M, N, K) >= 2 * M * N * 4, K
    assert size(fmt, anchors, M, N, 2048) == 0
    assert size("nf4", 0, M, N, 28672) >= 2 * M * N * 4 and size("nf4", 0, M, N, 8192) == 0


@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
def test_few_rows_and_short_sums_take_none(size, fmt):
    for M in (1, 4, 16, 32):
        assert size(fmt, 0, M, 500, 28672) == 0
    for M, N, K in ((333, 1501, 64), (48, 96, 512), (200, 96, 512), (40, 80, 4096)):
        assert size(fmt, 0, M, N, K) == 0, (M, N, K)
    assert size("2bit", 143, 40, 80, 4096) == 0
