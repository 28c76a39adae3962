"""qgemm_linear's kernels behind the large shapes, by their own choice and not by
a test hook: narrow tiles of many columns, column tiles of 256 and of 128 rows
beside each other, single rows that the decode GEMVs take. Against the formula in
64 bits, elementwise (bounds: layer_util.linear64)."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from layer_util import Matrix, activations, linear64
from routed_util import assert_close, tdt
from test_gpu_linear import case

pytestmark = pytest.mark.gpu

FORMS = [("2bit", 0), ("2bit", 21), ("nf4", 0), ("int4", 0), ("int4", 13)]


@pytest.mark.parametrize("fmt,anchors", FORMS)
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3", "i8"])
@pytest.mark.parametrize("M,N,gated", [(3, 17002, False), (4, 17002, True), (2, 10002, False), (9, 9602, True), (9, 12001, False),
                                       (16, 20002, False), (12, 20002, True), (24, 9601, False), (32, 12002, True)])
def test_narrow_tiles_of_many_columns(fmt, anchors, kind, M, N, gated):
    """Tiles of 4, 16 and 32 rows by 32 and 64 columns, 4 to 16 waves; columns past the last tile's end."""
    case(fmt, M, 320, N, kind, "f32", anchors, "f32", "silu" if gated else None, gated, "bf16", seed=M + N, rounded=False)


@pytest.mark.parametrize("fmt,anchors", FORMS)
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3", "i8"])
@pytest.mark.parametrize("M", [65, 128, 200])
def test_more_rows_by_narrow_tiles_round_no_weight(fmt, anchors, kind, M):
    case(fmt, M, 512, 96, kind, "f32", anchors, "f16", "relu", False, "f32", seed=M, rounded=False)


@pytest.mark.parametrize("fmt,anchors,kind,gated,act,bias,residual,y", [
    ("2bit", 9, "bf16", False, "relu", "bf16", "bf16", "bf16"), ("2bit", 70, "i8", True, "silu", "f32", "f16", "f16"),
    ("2bit", 0, "f16", False, None, "f16", "f32", "f32"), ("nf4", 0, "bf16", True, "silu", None, "bf16", "bf16"),
    ("nf4", 0, "e4m3", False, "silu", "f16", None, "bf16"), ("int4", 9, "e4m3", False, "relu", None, "f16", "f16"),
    ("int4", 66, "bf16", True, "silu", "bf16", "f32", "f32")])
def test_high_and_low_tiles_side_by_side(fmt, anchors, kind, gated, act, bias, residual, y):
    """4090 rows by 20 column tiles: 16 of them by 256 rows, which is one round of the
    CUs, the others by 128. Rows at the tiles' borders and ends, all columns; and
    in place of the residual."""
    import torch
    M, K, N = 4090, 192, 5118 if gated else 5117
    width = N // 2 if gated else N
    m = Matrix(fmt, N, K, anchors, 80)
    X, xs, x64 = activations(M, K, kind, 81)
    g = torch.Generator().manual_seed(82)
    b = (0.5 * torch.randn(N, generator=g)).to(tdt(bias)) if bias else None
    r = torch.randn(M, width, generator=g).to(tdt(residual)) if residual else None
    got = qw.qgemm_linear(m.pw, X, bias=b.cuda() if bias else None, act=act, gated=gated, residual=r.cuda() if residual else None,
                          x_scales=xs, out_dtype=tdt(y))
    for lo, hi in ((0, 36), (120, 136), (250, 262), (2040, 2056), (3960, M)):
        want, tol = linear64(m, x64[lo:hi], kind, True, b.double().numpy() if bias else None, act, gated,
                             r[lo:hi].double().numpy() if residual else None)
        assert_close(got[lo:hi], want, tol, tdt(y), f"rows {lo}")
    if residual == y:
        out = r.cuda()
        qw.qgemm_linear(m.pw, X, bias=b.cuda() if bias else None, act=act, gated=gated, residual=out, x_scales=xs, out=out)
        assert torch.equal(out, got)


@pytest.mark.parametrize("fmt,anchors", FORMS)
@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("K", [512, 1024, 576])
def test_few_fp16_rows_with_infinities_stay_alone(fmt, anchors, M, K):
    """An infinity or a NaN, at an anchor channel and at another, leaves nothing finite
    in its row, by the decode GEMVs too; the other rows keep their bits."""
    import torch
    m = Matrix(fmt, 100, K, anchors, 90)
    X, _, _ = activations(M, K, "f16", 91)
    clean = qw.qgemm_linear(m.pw, X, out_dtype=torch.float32)
    idx = m.pw.out_idx.cpu().numpy()[:anchors] if fmt == "2bit" and anchors else np.arange(anchors)
    other = next(c for c in range(K - 1, 0, -1) if c not in idx)
    for at in [other] + ([int(idx[0])] if anchors else []):
        for bad in (float("inf"), float("-inf"), float("nan")):
            Y = X.clone()
            Y[M - 1, at] = bad
            y = qw.qgemm_linear(m.pw, Y, out_dtype=torch.float32)
            assert torch.equal(y[: M - 1], clean[: M - 1])
            assert not bool(torch.isfinite(y[M - 1]).any()), (at, bad, int(torch.isfinite(y[M - 1]).sum()))
