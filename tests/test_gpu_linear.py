"""qgemm_linear against the formula in 64 bits, elementwise (the bounds are
derived in layer_util.linear64)."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from layer_util import Matrix, activations, linear64
from routed_util import assert_close, tdt

pytestmark = pytest.mark.gpu

ANCHORS = {"2bit": 0.035, "nf4": 0.0, "int4": 0.01}


def case(fmt, M, K, N, kind, y, n_out=None, bias=None, act=None, gated=False, residual=None, seed=0, rounded=False, ws=None):
    import torch
    n_out = int(ANCHORS[fmt] * K) if n_out is None else n_out
    m = Matrix(fmt, N, K, n_out, seed)
    X, xs, x64 = activations(M, K, kind, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    width = N // 2 if gated else N
    b = (0.5 * torch.randn(N, generator=g)).to(tdt(bias)) if bias else None
    r = torch.randn(M, width, generator=g).to(tdt(residual)) if residual else None
    got = qw.qgemm_linear(m.pw, X, bias=b.cuda() if bias else None, act=act, gated=gated, residual=r.cuda() if residual else None,
                          x_scales=xs, out_dtype=tdt(y), workspace=ws)
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
