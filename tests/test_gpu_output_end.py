"""GPU: outputs that end within the last 16 bytes below 2 GiB, where the
kernels still take byte offsets of 32 bits: the rows past a short tile and
the columns past N, which are dropped there, must not reach the last row."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from routed_util import F32, Experts, assert_close, half_step

pytestmark = pytest.mark.gpu

# n * N elements of 2 (4) bytes: 2^31 - 2 (2^31 - 4) bytes, N odd
SIZES = [("bf16", 360437, 2979), ("f32", 256999, 2089)]


def check(Y, x, ex, n, what):
    """The first row tile, the last rows, and every row's last columns."""
    import torch
    dt = Y.dtype
    w = torch.from_numpy(ex.W[0]).cuda()
    m = torch.from_numpy(ex.mag[0]).cuda()
    rows = torch.cat([torch.arange(300), torch.arange(n - 600, n)]).cuda()
    for r, c in ((rows, slice(0, ex.N)), (slice(0, n), slice(ex.N - 8, ex.N))):
        xr = x[r].double()
        want, mag = xr @ w[c].t(), xr.abs() @ m[c].t()
        tol = ((ex.K + 64) * F32 + half_step(torch.bfloat16) + F32) * mag
        assert_close(Y[r][:, c], want.cpu().numpy(), tol.cpu().numpy(), dt, what)


@pytest.mark.parametrize("out,n,N", SIZES)
@pytest.mark.parametrize("blocks", [1, 4, 8, 16])
@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
def test_experts(fmt, blocks, out, n, N, tune):
    import torch
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    ex = Experts(fmt, 1, N, 64, 0, seed=2)
    assert 2**31 - 16 < n * N * (2 if out == "bf16" else 4) < 2**31
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(n, 64, generator=gen, device="cuda").to(torch.bfloat16)
    g = qw.RowGroups(torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"))
    Y = qw.qgemm_experts(ex.ew, x, g, out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    check(Y, x, ex, n, f"{fmt} {blocks}")


@pytest.mark.parametrize("out,n,N", SIZES)
@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
@pytest.mark.parametrize("wide", [None, 0])
def test_prefill(fmt, out, n, N, wide, tune):
    import torch
    if wide is not None:
        tune(qw.QW_TUNE_PREFILL_WIDE_TILES, wide)
    ex = Experts(fmt, 1, N, 64, 0, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.randn(n, 64, generator=gen, device="cuda").to(torch.bfloat16)
    Y = qw.qgemm_prefill(ex.packed[0], x, out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    check(Y, x, ex, n, f"prefill {fmt}")
