"""CPU checks of the calls whose rows take different matrices: every refusal
the header documents comes before any device work, the size queries answer
on the host, and the binding refuses what the library would read wrongly."""

import ctypes
import os

import pytest

from bit_weight_quantized_qw_amd import qw

P = 0x1000    # stands for a device address; nothing may touch it
ODD = 0x1004


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qw.LIB_PATH):
        from bit_weight_quantized_qw_amd.build import build
        build()
    return qw.lib()


def groups(G=4, n=8, off=P, rows=P):
    return ctypes.byref(qw.qw_groups(G, n, off, rows))


def experts(E=4, fmt=qw.QW_FMT_2BIT_G32, N=16, K=64, n_out=0, codes=P, **kw):
    pad = (n_out + 7) // 8 * 8
    w = qw.qw_weight(fmt, N, K, n_out, pad, codes, kw.get("scales", P), kw.get("idx", P if n_out else None),
                     kw.get("wo", P if n_out else None), kw.get("mask", P if n_out else None))
    return ctypes.byref(qw.qw_experts(E, w))


F16, BF16, F32 = qw.QW_DT_F16, qw.QW_DT_BF16, qw.QW_DT_F32
INV, ALIGN, UNSUP = qw.QW_ERR_INVALID_ARG, qw.QW_ERR_ALIGNMENT, qw.QW_ERR_UNSUPPORTED


def test_group_rows_refusals(L):
    def call(ids=P, n=8, G=4, off=P, rows=P, ws=P, nb=1 << 20):
        return L.qw_group_rows(ids, n, G, off, rows, ws, nb, None)
    for kw in ({"ids": None}, {"off": None}, {"rows": None}, {"n": 0}, {"n": -1}, {"G": 0}):
        assert call(**kw) == INV, kw
    for kw in ({"ids": ODD}, {"off": ODD}, {"rows": ODD}, {"n": 10000, "ws": ODD}):
        assert call(**kw) == ALIGN, kw
    assert call(G=qw.QW_MAX_GROUPS + 1) == UNSUP
    assert call(n=qw.QW_MAX_ROWS + 1) == UNSUP
    need = qw.qw_group_rows_workspace_bytes(10000, 4)
    assert need > 0 and call(n=10000, nb=need - 1) == INV and call(n=10000, ws=None, nb=need) == INV
    assert qw.qw_group_rows_workspace_bytes(100, 4) == 0
    assert qw.qw_group_rows_workspace_bytes(0, 4) == qw.qw_group_rows_workspace_bytes(10, 0) == 0
    assert qw.qw_group_rows_workspace_bytes(10000, qw.QW_MAX_GROUPS + 1) == 0


def test_route_refusals(L):
    def call(x=P, dt=F32, T=4, E=8, k=2, ids=P, w=P, off=P, rows=P, ws=P, nb=1 << 24):
        return L.qw_route_topk(x, dt, T, E, k, 1, ids, w, off, rows, ws, nb, None)
    for kw in ({"x": None}, {"ids": None}, {"w": None}, {"off": None}, {"rows": None}, {"T": 0}, {"E": 0}, {"k": 0},
               {"k": 9}, {"dt": 0}, {"dt": 9}, {"E": 64, "k": qw.QW_MAX_TOPK + 1}):
        assert call(**kw) == INV, kw
    for kw in ({"x": ODD}, {"ids": ODD}, {"w": ODD}, {"off": ODD}, {"rows": ODD}, {"T": 4000, "ws": ODD}):
        assert call(**kw) == ALIGN, kw
    assert call(E=qw.QW_MAX_GROUPS + 1) == UNSUP
    assert call(T=qw.QW_MAX_ROWS, k=2) == UNSUP
    need = qw.qw_route_workspace_bytes(4000, 8, 2)
    assert need > 0 and call(T=4000, nb=need - 1) == INV and call(T=4000, ws=None) == INV
    assert qw.qw_route_workspace_bytes(48, 64, 8) == 0
    assert qw.qw_route_workspace_bytes(48, 4, 8) == 0  # top_k > E


def test_experts_refusals(L):
    def call(ew=None, X=P, dt=F16, x_rows=8, div=1, g=None, sw=0, Y=P, ydt=F16):
        return L.qgemm_experts(ew or experts(), X, dt, x_rows, div, g or groups(), sw, Y, ydt, None)
    assert L.qgemm_experts(None, P, F16, 8, 1, groups(), 0, P, F16, None) == INV
    assert L.qgemm_experts(experts(), P, F16, 8, 1, None, 0, P, F16, None) == INV
    for kw in ({"X": None}, {"Y": None}, {"dt": F32}, {"dt": 0}, {"ydt": 0}, {"x_rows": 0}, {"div": -1},
               {"div": 0, "x_rows": 7}, {"ew": experts(E=0)}, {"ew": experts(E=5)}, {"ew": experts(fmt=9)},
               {"ew": experts(codes=None)}, {"ew": experts(K=48)}, {"ew": experts(N=0)}, {"ew": experts(n_out=3, idx=None)},
               {"ew": experts(n_out=3, mask=None)}, {"ew": experts(n_out=3, wo=None)},
               {"ew": experts(fmt=qw.QW_FMT_NF4_B64, n_out=3)}, {"g": groups(G=0)}, {"g": groups(n=0)},
               {"g": groups(off=None)}, {"g": groups(rows=None)}, {"sw": 1, "ew": experts(N=17)}):
        assert call(**kw) == INV, kw
    for kw in ({"X": ODD}, {"Y": ODD}, {"ew": experts(codes=ODD)}, {"ew": experts(scales=ODD)}, {"g": groups(off=ODD)},
               {"g": groups(rows=ODD)}):
        assert call(**kw) == ALIGN, kw
    assert call(ew=experts(K=96)) == UNSUP
    assert call(ew=experts(N=1 << 20, K=1 << 12)) == UNSUP
    big = qw.QW_MAX_GROUPS + 1
    assert call(ew=experts(E=big), g=groups(G=big)) == UNSUP
    assert call(g=groups(n=qw.QW_MAX_ROWS + 1), x_rows=1 << 25) == UNSUP


def test_combine_refusals(L):
    need = qw.qw_experts_combine_workspace_bytes(16, 4, 2)
    assert need == 4 * 2 * 16 * 4

    def call(ew=None, H=P, dt=F16, g=None, ids=P, w=P, T=4, k=2, out=P, odt=F16, ws=P, nb=need):
        return L.qgemm_experts_combine(ew or experts(), H, dt, g or groups(), ids, w, T, k, out, odt, ws, nb, None)
    for kw in ({"H": None}, {"ids": None}, {"w": None}, {"out": None}, {"T": 0}, {"k": 0}, {"T": 3}, {"k": 3}, {"dt": F32},
               {"odt": 0}, {"ws": None}, {"nb": need - 1}, {"ew": experts(E=5)}):
        assert call(**kw) == INV, kw
    for kw in ({"H": ODD}, {"ids": ODD}, {"w": ODD}, {"out": ODD}, {"ws": ODD}):
        assert call(**kw) == ALIGN, kw
    assert call(ew=experts(K=96)) == UNSUP
    assert qw.qw_experts_combine_workspace_bytes(0, 4, 2) == qw.qw_experts_combine_workspace_bytes(16, 0, 2) == 0
    assert qw.qw_experts_combine_workspace_bytes(16, qw.QW_MAX_ROWS, 2) == 0
    assert qw.qw_experts_combine_workspace_bytes(1 << 20, 1 << 20, 4) == (1 << 42) * 4


def adapters(count=4, N=16, K=64, r=8, dt=F16, A=P, B=P, scale=P):
    return ctypes.byref(qw.qw_adapters(count, N, K, r, dt, A, B, scale))


def test_lora_refusals(L):
    need = L.qw_lora_workspace_bytes(adapters(), 8)
    assert need == 8 * 8 * 4

    def call(ad=None, x=P, g=None, base=P, bdt=F16, out=P, odt=F16, ws=P, nb=need):
        return L.qw_lora_add(ad or adapters(), x, g or groups(), base, bdt, out, odt, ws, nb, None)
    assert L.qw_lora_add(None, P, groups(), P, F16, P, F16, P, need, None) == INV
    for kw in ({"x": None}, {"base": None}, {"out": None}, {"bdt": 0}, {"odt": 9}, {"odt": F32}, {"ws": None}, {"nb": need - 1},
               {"ad": adapters(count=0)}, {"ad": adapters(count=5)}, {"ad": adapters(N=0)}, {"ad": adapters(K=60)},
               {"ad": adapters(r=12)}, {"ad": adapters(r=0)}, {"ad": adapters(dt=F32)}, {"ad": adapters(A=None)},
               {"ad": adapters(B=None)}, {"ad": adapters(scale=None)}, {"g": groups(n=0)}, {"g": groups(rows=None)}):
        assert call(**kw) == INV, kw  # odt F32 on the address of an fp16 base: in place with another type
    for kw in ({"x": ODD}, {"base": ODD}, {"out": ODD}, {"ws": ODD}, {"ad": adapters(A=ODD)}, {"ad": adapters(B=ODD)},
               {"ad": adapters(scale=ODD)}):
        assert call(**kw) == ALIGN, kw
    assert call(ad=adapters(r=qw.QW_MAX_RANK + 8), nb=1 << 30) == UNSUP
    assert L.qw_lora_workspace_bytes(adapters(r=12), 8) == L.qw_lora_workspace_bytes(adapters(), 0) == 0
    assert L.qw_lora_workspace_bytes(None, 8) == 0


def test_tuning_hook(L):
    assert qw.qw_tune_get(qw.QW_TUNE_EXPERTS_ROW_BLOCKS) == qw.QW_TUNE_AUTO
    with qw.tuned(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, 4):
        assert qw.qw_tune_get(qw.QW_TUNE_EXPERTS_ROW_BLOCKS) == 4


def test_valid_calls_without_gpu_report_no_device(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert L.qw_group_rows(P, 8, 4, P, P, None, 0, None) == qw.QW_ERR_NO_DEVICE
    assert L.qw_route_topk(P, F32, 4, 8, 2, 1, P, P, P, P, None, 0, None) == qw.QW_ERR_NO_DEVICE
    assert L.qgemm_experts(experts(), P, F16, 8, 1, groups(), 0, P, F16, None) == qw.QW_ERR_NO_DEVICE
    assert L.qw_lora_add(adapters(), P, groups(), P, F16, P, F16, P, 1 << 20, None) == qw.QW_ERR_NO_DEVICE


def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(TypeError):
        qw.RowGroups(torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        qw.qw_group_rows(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(TypeError):
        qw.qw_route_topk(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError):
        qw.Adapters(torch.zeros(2, 8, 64).half(), torch.zeros(2, 16, 8).half(), torch.zeros(2))
    with pytest.raises(ValueError):
        qw.ExpertWeights(qw.QW_FMT_2BIT_G32, 2, 16, 64, codes=torch.zeros(512, dtype=torch.uint8),
                         scales=torch.zeros(256, dtype=torch.uint8))
