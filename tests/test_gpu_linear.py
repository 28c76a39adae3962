"""qgemm_linear against the formula in 64 bits, elementwise (the bounds are
derived in layer_util.linear64)."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from layer_util import Matrix, activations, linear64
from routed_util import assert_close, tdt

pytestmark = pytest.mark.gpu

ANCHORS = {"2bit": 0.035, "nf4": 0.0, "int4": 0.01}


def case(fmt, M, K, N, kind, y, n_out=None, bias=None, act=None, gated=False, residual=None, seed=0, rounded=None):
    import torch
    n_out = int(ANCHORS[fmt] * K) if n_out is None else n_out
    rounded = M > 64 if rounded is None else rounded  # tall tiles from 65 rows on, if at all
    m = Matrix(fmt, N, K, n_out, seed)
    X, xs, x64 = activations(M, K, kind, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    width = N // 2 if gated else N
    b = (0.5 * torch.randn(N, generator=g)).to(tdt(bias)) if bias else None
    r = torch.randn(M, width, generator=g).to(tdt(residual)) if residual else None
    got = qw.qgemm_linear(m.pw, X, bias=b.cuda() if bias else None, act=act, gated=gated, residual=r.cuda() if residual else None,
                          x_scales=xs, out_dtype=tdt(y))
    want, tol = linear64(m, x64, kind, rounded, b.double().numpy() if bias else None, act, gated,
                         r.double().numpy() if residual else None)
    assert got.dtype == tdt(y) and tuple(got.shape) == (M, width)
    assert_close(got, want, tol, tdt(y), f"{fmt} {kind} {M}x{K}x{N}")


@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3", "i8"])
@pytest.mark.parametrize("anchors", [False, True])
@pytest.mark.parametrize("M", [1, 5, 33])
def test_types(fmt, kind, anchors, M):
    if anchors and fmt == "nf4":
        pytest.skip("NF4 has no anchors")
    case(fmt, M, 640, 200, kind, "f32", None if anchors else 0)


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("bias,residual", [(None, None), ("f16", None), (None, "f32"), ("f32", "bf16"), ("bf16", "f16")])
def test_epilogues(act, gated, bias, residual):
    case("int4", 19, 512, 136, "bf16", "f32", 5, bias, act, gated, residual, seed=3)


@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
@pytest.mark.parametrize("y", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("N", [2, 30, 64, 66, 130, 258, 500])
def test_odd_columns_and_output_types(fmt, y, N):
    for gated in (False, True):
        case(fmt, 3, 192, N, "f16", y, bias=y, act="silu", gated=gated, residual=y, seed=N)
    case(fmt, 18, 192, N + 1, "e4m3", y, bias=y, residual="f32", seed=N)


@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
@pytest.mark.parametrize("K", [64, 128, 320, 1024, 2112, 4096])
def test_lengths_of_the_sums(fmt, K):
    case(fmt, 2, K, 80, "bf16", "f32", seed=K)
    case(fmt, 40, K, 80, "i8", "f32", seed=K)


@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
@pytest.mark.parametrize("M", [1, 2, 4, 15, 16, 17, 31, 32, 48, 64, 65, 100, 128, 129, 200])
def test_rows(fmt, M):
    case(fmt, M, 512, 96, "f16", "f32", seed=M)


# every kernel on the same shapes: 16-row blocks of a tile (4: four rows), parts of K
PATHS = [(4, 1), (4, 2), (1, 1), (1, 3), (2, 1), (2, 4), (8, 1), (8, 3), (16, 1), (16, 2)]


@pytest.mark.parametrize("blocks,parts", PATHS)
@pytest.mark.parametrize("fmt,anchors", [("2bit", 0), ("2bit", 37), ("nf4", 0), ("int4", 0), ("int4", 70)])
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3", "i8"])
def test_every_kernel(tune, blocks, parts, fmt, anchors, kind):
    """K of five steps of 64 (an odd number, uneven parts), rows and columns past a tile's end."""
    tune(qw.QW_TUNE_LINEAR_ROW_BLOCKS, blocks)
    tune(qw.QW_TUNE_LINEAR_PARTS, parts)
    case(fmt, 130, 832, 300, kind, "f32", anchors, seed=blocks + 20 * parts, rounded=blocks >= 8)


@pytest.mark.parametrize("blocks,parts", PATHS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N", [258, 516, 600])
def test_every_kernel_and_epilogue(tune, blocks, parts, gated, N):
    """Odd numbers of columns and of pairs, every epilogue part, each output type."""
    tune(qw.QW_TUNE_LINEAR_ROW_BLOCKS, blocks)
    tune(qw.QW_TUNE_LINEAR_PARTS, parts)
    for y in ("f16", "bf16", "f32"):
        case("int4", 100, 512, N, "bf16", y, 9, "f32", "silu", gated, "bf16", seed=N, rounded=blocks >= 8)
    case("2bit", 270, 320, N + (0 if gated else 1), "i8", "f16", 11, "f16", "gelu", gated, "f16", seed=N + 1, rounded=blocks >= 8)


@pytest.mark.parametrize("fmt,anchors", [("2bit", 0), ("2bit", 40), ("nf4", 0), ("int4", 0), ("int4", 9)])
@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K", [(1000, 512), (5120, 1024), (30, 2560), (11000, 512), (9000, 576)])
def test_few_rows_fp16(fmt, anchors, M, N, K):
    """Single tokens: the decode GEMVs' shapes and those that they do not take, with every
    epilogue part."""
    case(fmt, M, K, N, "f16", "f32", anchors, "f16", "gelu_tanh", False, "bf16", seed=M + N)
    case(fmt, M, K, N, "f16", "f16", anchors, None, None, False, "f16", seed=M + N)
    case(fmt, M, K, N, "f16", "f16", anchors, "f32", "silu", True, "f32", seed=M + N)


def test_fp16_weights_of_any_size_keep_their_bits(tune):
    """Tall tiles with fp16 activations: scales of 1e-6 and of 1e4, anchors larger
    than the rest of their column."""
    import torch
    tune(qw.QW_TUNE_LINEAR_ROW_BLOCKS, 8)
    X, _, x64 = activations(40, 256, "f16", 31)
    for fmt, n_out in (("2bit", 9), ("int4", 9), ("nf4", 0)):
        for size in (1e-6, 1.0, 1e4):
            m = Matrix(fmt, 64, 256, n_out, 30)
            if fmt == "nf4":
                m.pw.scales.view(torch.float32).mul_(size)
                m.W1, m.mag1 = m.W1 * np.float64(np.float32(size)), m.mag1 * size
                extra = 2.0 ** -23  # the product with size, rounded
            elif size < 1:
                continue  # an fp16 Z would lose bits below 2^-14
            else:  # fp16 scales: times a power of two, which is exact
                size = 2.0 ** 10 if size > 1 else 1.0
                m.pw.scales.view(torch.float16).mul_(size)
                big = m.pw.out_w.view(torch.float16)
                big.mul_(64.0)
                idx = m.pw.out_idx.cpu().numpy()[:n_out] if fmt == "2bit" else np.arange(n_out)
                keep = np.ones(256, bool)
                keep[idx] = False
                m.W1[:, keep] *= size
                m.mag1[:, keep] *= size
                m.W1[:, idx] *= 64
                m.mag1[:, idx] *= 64
                extra = 0.0
            got = qw.qgemm_linear(m.pw, X, out_dtype=torch.float32)
            want, tol = linear64(m, x64, "f16", True)
            assert_close(got, want, tol + extra * (np.abs(x64) @ m.mag1.T), torch.float32, f"{fmt} {size}")


def test_gated_bf16_rows_of_any_size(tune):
    """Tall gated tiles: rows of 1e-30, 1e30, zeros and one with an infinity, one large channel."""
    import torch
    tune(qw.QW_TUNE_LINEAR_ROW_BLOCKS, 8)
    m = Matrix("int4", 128, 256, 5, 50)
    X, _, _ = activations(40, 256, "bf16", 51)
    X[0] *= 1e-30
    X[1] *= 1e8
    X[2] = 0
    X[3, 7] = float("inf")
    X[4, 9] = 3e4
    x64 = X.double().cpu().numpy()
    y = qw.qgemm_linear(m.pw, X, gated=True, out_dtype=torch.float32)
    keep = [i for i in range(40) if i != 3]
    want, tol = linear64(m, x64[keep], "bf16", True, gated=True)
    assert_close(y[keep], want, tol, torch.float32)
    assert bool((y[2] == 0).all()) and not bool(torch.isfinite(y[3]).any())


def test_gated_bf16_infinity_beside_large_numbers(tune):
    """Tall gated tiles: one infinity among numbers past fp16's range gives infinities of
    the weights' signs, not NaN."""
    import torch
    tune(qw.QW_TUNE_LINEAR_ROW_BLOCKS, 8)
    m = Matrix("nf4", 128, 256, 0, 52)
    X = torch.full((40, 256), 1e6, dtype=torch.bfloat16, device="cuda")
    X[3, 7] = float("inf")
    y = qw.qgemm_linear(m.pw, X, gated=True, out_dtype=torch.float32)[3].cpu().numpy()
    sign = np.sign(m.W1[:64, 7]) * np.sign(m.W1[64:, 7])  # no weight: infinity times 0
    assert (sign != 0).sum() > 30
    assert (y[sign != 0] == np.inf * sign[sign != 0]).all() and np.isnan(y[sign == 0]).all()


@pytest.mark.parametrize("fmt", ["2bit", "nf4", "int4"])
@pytest.mark.parametrize("gated", [False, True])
def test_one_step_of_K_and_more_rows_than_a_launch_of_narrow_tiles(fmt, gated):
    """K of 64 by 2^20 + 3 rows and 17000 columns, 70 million waves of narrow tiles: the rows at both ends."""
    import torch
    M, N = (1 << 20) + 3, 17000
    m = Matrix(fmt, N, 64, 0, 53)
    X = torch.randn(M, 64, device="cuda").half()
    y = qw.qgemm_linear(m.pw, X, gated=gated, out_dtype=torch.float16)
    for rows in (slice(0, 40), slice(M - 40, M)):
        want, tol = linear64(m, X[rows].double().cpu().numpy(), "f16", True, gated=gated)
        assert_close(y[rows], want, tol, torch.float16)


def test_rows_do_not_depend_on_each_other_and_ends_stay():
    """A row's values do not change with its place; nothing is written behind Y."""
    import torch
    m = Matrix("2bit", 70, 256, 9, 5)
    X, _, _ = activations(20, 256, "f16", 6)
    y = qw.qgemm_linear(m.pw, X)
    turn = torch.randperm(20, device="cuda")
    assert torch.equal(y[turn], qw.qgemm_linear(m.pw, X[turn].contiguous()))
    buf = torch.full((20 * 70 + 64,), 7.0, dtype=torch.float16, device="cuda")
    out = buf[: 20 * 70].view(20, 70)
    assert torch.equal(qw.qgemm_linear(m.pw, X, out=out), y) and bool((buf[20 * 70:] == 7).all())


def test_residual_in_place():
    import torch
    m = Matrix("nf4", 90, 128, 0, 7)
    X, _, _ = activations(35, 128, "bf16", 8)
    r = torch.randn(35, 90, device="cuda").bfloat16()
    want = qw.qgemm_linear(m.pw, X, residual=r)
    assert torch.equal(qw.qgemm_linear(m.pw, X, residual=r, out=r), want)


def test_rows_with_infinities_stay_alone():
    import torch
    m = Matrix("int4", 50, 256, 0, 9)
    X, _, _ = activations(20, 256, "f16", 10)
    clean = qw.qgemm_linear(m.pw, X, act="relu")
    X[3, 5], X[18, 200] = float("inf"), float("nan")
    y = qw.qgemm_linear(m.pw, X, act="relu")
    keep = [i for i in range(20) if i not in (3, 18)]
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[18]).all())


def test_large_arguments_of_the_activations():
    """exp and erfc beyond their ranges: act(z) goes to z and to 0, never to NaN."""
    import torch
    m = Matrix("nf4", 64, 64, 0, 11)
    X = torch.full((1, 64), 1.0, device="cuda").half()
    b = torch.linspace(-300, 300, 64).cuda()
    z = qw.qgemm_linear(m.pw, X, bias=b, out_dtype=torch.float32)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        y = qw.qgemm_linear(m.pw, X, bias=b, act=act, out_dtype=torch.float32)
        assert bool(torch.isfinite(y).all())
        assert torch.equal(y[0, 40:], z[0, 40:]) and float(y[0, :20].abs().max()) < 1e-30


def test_refusals_of_the_binding():
    import torch
    m = Matrix("2bit", 16, 64, 0, 12)
    X = torch.zeros(4, 64, device="cuda").half()
    s = torch.ones(4, device="cuda")
    for kw in ({"act": "tanh"}, {"x_scales": s}, {"bias": torch.zeros(15, device="cuda")}, {"residual": torch.zeros(4, 15, device="cuda")},
               {"residual": torch.zeros(4, 16, device="cuda"), "gated": True}, {"out": torch.zeros(4, 17, device="cuda").half()}):
        with pytest.raises(ValueError):
            qw.qgemm_linear(m.pw, X, **kw)
    with pytest.raises(ValueError):
        qw.qgemm_linear(m.pw, X.to(torch.int8))
    with pytest.raises(ValueError):
        qw.qgemm_linear(m.pw, X.to(torch.int8), x_scales=s[:3])
    with pytest.raises(ValueError):
        qw.qgemm_linear(m.pw, X[:, :32].contiguous())
    with pytest.raises(ValueError):
        qw.qgemm_linear(m.pw, torch.zeros(64, 4, device="cuda").half().t())
    with pytest.raises(TypeError):
        qw.qgemm_linear(m.pw, X.float())
    y = torch.zeros(4, 16, device="cuda")
    with pytest.raises(qw.QwError):  # in place, but of another type
        qw.qgemm_linear(m.pw, X, residual=y, out=y.view(torch.float16).view(-1)[:64].view(4, 16))
