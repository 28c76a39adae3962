"""CPU checks of the calls around a projection (norm, product with epilogue,
router by scores): every refusal the header documents comes before any device
work, the size queries answer on the host, and the binding refuses what the
library would read wrongly."""

import ctypes
import os

import pytest

from bit_weight_quantized_qw_amd import qw

P = 0x1000    # stands for a device address; nothing may touch it
ODD = 0x1004
F16, BF16, F32, E4M3, I8 = qw.QW_DT_F16, qw.QW_DT_BF16, qw.QW_DT_F32, qw.QW_DT_E4M3, qw.QW_DT_I8
INV, ALIGN, UNSUP = qw.QW_ERR_INVALID_ARG, qw.QW_ERR_ALIGNMENT, qw.QW_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qw.LIB_PATH):
        from bit_weight_quantized_qw_amd.build import build
        build()
    return qw.lib()


def test_rmsnorm_refusals(L):
    def call(x=P, xdt=F16, r=None, rdt=0, w=P, wdt=F16, eps=1e-6, M=4, K=64, perm=None, ro=None, y=P, ydt=F16, sc=None):
        return L.qw_rmsnorm(x, xdt, r, rdt, w, wdt, eps, M, K, perm, ro, y, ydt, sc, None)
    for kw in ({"x": None}, {"w": None}, {"y": None}, {"M": 0}, {"K": 0}, {"M": -1}, {"xdt": 0}, {"xdt": E4M3}, {"xdt": 6},
               {"wdt": I8}, {"r": P}, {"r": P, "rdt": E4M3}, {"ro": P}, {"ydt": 0}, {"ydt": 6}, {"ydt": E4M3}, {"ydt": I8},
               {"sc": P}, {"eps": -1e-6}, {"eps": float("nan")}, {"eps": float("inf")}):
        assert call(**kw) == INV, kw
    for kw in ({"x": ODD}, {"w": ODD}, {"y": ODD}, {"r": ODD, "rdt": F16}, {"r": P, "rdt": F16, "ro": ODD}, {"perm": ODD},
               {"ydt": I8, "sc": ODD}):
        assert call(**kw) == ALIGN, kw
    assert call(K=qw.QW_MAX_NORM_K + 1) == UNSUP
    assert call(M=qw.QW_MAX_ROWS + 1) == UNSUP


def weight(fmt=qw.QW_FMT_2BIT_G32, N=16, K=64, n_out=0, codes=P, **kw):
    pad = (n_out + 7) // 8 * 8
    return ctypes.byref(qw.qw_weight(fmt, N, K, n_out, pad, codes, kw.get("scales", P), kw.get("idx", P if n_out else None),
                                     kw.get("wo", P if n_out else None), kw.get("mask", P if n_out else None)))


def epilogue(**kw):
    return ctypes.byref(qw.qw_epilogue(**kw))


def test_linear_refusals(L):
    def call(w=None, X=P, dt=F16, xs=None, M=4, ep=None, Y=P, ydt=F16, ws=P, nb=1 << 30):
        return L.qgemm_linear(w or weight(), X, dt, xs, M, ep, Y, ydt, ws, nb, None)
    assert L.qgemm_linear(None, P, F16, None, 4, None, P, F16, None, 0, None) == INV
    for kw in ({"X": None}, {"Y": None}, {"M": 0}, {"dt": 0}, {"dt": F32}, {"dt": 6}, {"ydt": 0}, {"ydt": E4M3}, {"dt": E4M3},
               {"dt": I8}, {"xs": P}, {"dt": BF16, "xs": P}, {"w": weight(fmt=9)}, {"w": weight(codes=None)}, {"w": weight(K=48)},
               {"w": weight(N=0)}, {"w": weight(n_out=3, idx=None)}, {"w": weight(n_out=3, mask=None)},
               {"w": weight(n_out=3, wo=None)}, {"w": weight(fmt=qw.QW_FMT_NF4_B64, n_out=3)},
               {"ep": epilogue(act=-1)}, {"ep": epilogue(act=5)}, {"ep": epilogue(bias=P)}, {"ep": epilogue(bias=P, bias_dtype=I8)},
               {"ep": epilogue(residual=P)}, {"ep": epilogue(residual=P, residual_dtype=E4M3)},
               {"ep": epilogue(gated=1), "w": weight(N=17)},
               {"ep": epilogue(residual=P, residual_dtype=F32), "Y": P}):  # in place with another type
        assert call(**kw) == INV, kw
    for kw in ({"X": ODD}, {"Y": ODD}, {"dt": I8, "xs": ODD}, {"w": weight(codes=ODD)}, {"w": weight(scales=ODD)},
               {"ep": epilogue(bias=ODD, bias_dtype=F16)}, {"ep": epilogue(residual=ODD, residual_dtype=F16)}):
        assert call(**kw) == ALIGN, kw
    assert call(w=weight(K=96)) == UNSUP
    assert call(w=weight(N=1 << 20, K=1 << 12)) == UNSUP
    assert call(w=weight(N=4, K=1 << 22)) == UNSUP
    assert call(M=qw.QW_MAX_ROWS + 1) == UNSUP
    big = weight(N=4096, K=8192)
    need = L.qw_linear_workspace_bytes(big, F16, 100, 0)  # K in parts
    assert need >= 2 * 100 * 4096 * 4 and L.qw_linear_workspace_bytes(big, F16, 1, 0) == 0
    assert L.qw_linear_workspace_bytes(big, BF16, 3000, 1) >= 3000 * 8192 * 2  # the activations in fp16
    assert call(w=big, M=100, nb=need - 1) == INV and call(w=big, M=100, ws=None, nb=need) == INV
    assert call(w=big, M=100, ws=ODD, nb=need) == ALIGN
    size = L.qw_linear_workspace_bytes
    assert size(None, F16, 4, 0) == size(weight(), F16, 0, 0) == size(weight(N=17), BF16, 4000, 1) == 0
    assert size(weight(K=96), F16, 4, 0) == size(weight(fmt=9), F16, 4, 0) == 0


def test_route_scored_refusals(L):
    def call(x=P, dt=F32, T=4, E=8, k=2, sc=qw.QW_ROUTE_SIGMOID, b=None, n=2, top=1, by=qw.QW_GROUP_TOP2, f=1.0, ids=P, w=P,
             off=P, rows=P, ws=P, nb=1 << 24):
        return L.qw_route_scored(x, dt, T, E, k, sc, b, n, top, by, 1, f, ids, w, off, rows, ws, nb, None)
    for kw in ({"x": None}, {"ids": None}, {"w": None}, {"off": None}, {"rows": None}, {"T": 0}, {"E": 0}, {"k": 0}, {"k": 5},
               {"dt": 0}, {"dt": E4M3}, {"E": 128, "k": qw.QW_MAX_TOPK + 1}, {"sc": 0}, {"sc": 3}, {"by": 0}, {"by": 3}, {"n": 0},
               {"n": 3}, {"top": 0}, {"top": 3}, {"E": 130, "n": 65, "top": 65}, {"f": float("nan")}, {"f": float("inf")}):
        assert call(**kw) == INV, kw
    for kw in ({"x": ODD}, {"b": ODD}, {"ids": ODD}, {"w": ODD}, {"off": ODD}, {"rows": ODD}, {"T": 4000, "ws": ODD}):
        assert call(**kw) == ALIGN, kw
    assert call(E=2 * qw.QW_MAX_GROUPS) == UNSUP
    assert call(T=qw.QW_MAX_ROWS, k=2) == UNSUP
    need = qw.qw_route_scored_workspace_bytes(4000, 8, 2, 2)
    assert need > 0 and call(T=4000, nb=need - 1) == INV and call(T=4000, ws=None) == INV
    assert qw.qw_route_scored_workspace_bytes(8, 64, 8, 8) == 0
    assert qw.qw_route_scored_workspace_bytes(4000, 8, 2, 3) == qw.qw_route_scored_workspace_bytes(4000, 8, 9, 2) == 0


def test_valid_calls_without_gpu_report_no_device(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    none = qw.QW_ERR_NO_DEVICE
    assert L.qw_rmsnorm(P, F16, P, F32, P, F32, 1e-6, 4, 64, P, P, P, E4M3, P, None) == none
    assert L.qgemm_linear(weight(), P, I8, P, 4, epilogue(bias=P, bias_dtype=F16, residual=P, residual_dtype=F16, gated=1), P, F16,
                          P, 1 << 30, None) == none
    assert L.qgemm_linear(weight(), P, F16, None, 4, None, P, F32, P, 1 << 30, None) == none
    assert L.qw_route_scored(P, BF16, 4, 8, 4, qw.QW_ROUTE_SOFTMAX, P, 2, 1, qw.QW_GROUP_MAX, 0, 2.5, P, P, P, P, None, 0, None) == none


def test_binding_refuses_host_tensors_and_names():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        qw.qw_rmsnorm(x, torch.ones(64))
    with pytest.raises(TypeError):
        qw.qw_route_scored(x, 2)
    pw = type("W", (), {"N": 16, "K": 64})()
    with pytest.raises(TypeError):
        qw.qgemm_linear(pw, x.half())
