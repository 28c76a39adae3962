"""GPU: the experts' products over grouped rows (plain, gated, and summed per
token) against the dequantized weights in 64 bits, elementwise within the
bounds of routed_util."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import F32, Experts, assert_close, device_groups, gated, products, tdt

pytestmark = pytest.mark.gpu


def is_wide(n, E):
    """Whether the call may take the kernel of wide tiles (by itself it
    chooses by an estimate of the time, from several rows an expert on)."""
    forced = qw.qw_tune_get(qw.QW_TUNE_EXPERTS_ROW_BLOCKS)
    return forced > 1 if forced > 0 else n > 2 * E


def is_tall(n, ex, dt, odt, swiglu):
    """Whether it may take the kernel of tall tiles, whose weights are
    rounded to the activations' type."""
    import torch
    forced = qw.qw_tune_get(qw.QW_TUNE_EXPERTS_ROW_BLOCKS)
    fits = odt in (dt, torch.float32) and not swiglu and not ex.packed[0].n_out
    return fits and (forced >= 8 if forced > 0 else n > 8 * ex.E)


def acts(rng, rows, K, dt):
    import torch
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x[:, rng.integers(0, K, max(1, K // 50))] *= 8
    return to_dev(x).to(dt)


def ids_of(rng, T, k, E, none=0.1):
    """Distinct experts per token, some tokens without any, later experts rarer."""
    p = 1.0 / (1 + np.arange(E))
    ids = np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)
    ids[rng.random(T) < none] = -1
    return ids


def check(ex, T, k, dtype, out="f32", swiglu=False, seed=0, none=0.1, grouped=False, rounded=None):
    import torch
    rng = np.random.default_rng(seed)
    ids = ids_of(rng, T, k, ex.E, none)
    g, off, rows = device_groups(ids, ex.E)
    dt, odt = tdt(dtype), tdt(out)
    x = acts(rng, T * k if grouped else T, ex.K, dt)
    N = ex.N // 2 if swiglu else ex.N
    Y = torch.full((T * k, N), 7.0, dtype=odt, device="cuda")
    got = qw.qgemm_experts(ex.ew, x, g, top_k=None if grouped else k, swiglu=swiglu, out=Y)
    assert got is Y
    x64 = x.double().cpu().numpy()
    y, tol = products(ex, x64 if grouped else x64[rows // k], off, is_wide(T * k, ex.E), dt,
                      is_tall(T * k, ex, dt, odt, swiglu))
    if swiglu:
        y, tol = gated(y, tol)
    m = off[-1]
    assert_close(Y[:m], y[:m], tol[:m], odt, f"{ex.fmt} {T}x{k} {dtype}->{out}")
    assert bool((Y[m:] == 7.0).all()), "rows of no group were written"


FORMATS = [("2bit", 0), ("2bit", 9), ("nf4", 0), ("int4", 0), ("int4", 5)]


@pytest.mark.parametrize("fmt,n_out", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N,K", [(1, 64), (17, 128), (64, 256), (70, 320), (129, 576), (200, 1088)])
def test_few_rows(fmt, n_out, dtype, N, K):
    """Shapes that end inside a tile of columns, a run of 64 weights or a
    quarter of K, for one token and for some."""
    ex = Experts(fmt, 5, N, K, n_out, seed=N + K)
    for T, k in ((1, 1), (1, 3), (7, 2), (30, 4)):
        check(ex, T, k, dtype, seed=T)
        check(ex, T, k, dtype, out=dtype, seed=T + 50)


@pytest.mark.parametrize("fmt,n_out", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N,K", [(40, 192), (260, 448), (300, 1024)])
@pytest.mark.parametrize("blocks", [None, 1, 2, 4, 8, 16])
def test_many_rows(fmt, n_out, dtype, N, K, blocks, tune):
    """Some hundred rows an expert, unevenly, by every tile height."""
    if blocks:
        tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    ex = Experts(fmt, 3, N, K, n_out, seed=N)
    for T, k in ((48, 2), (331, 2), (701, 1)):
        check(ex, T, k, dtype, seed=T)
        check(ex, T, k, dtype, out=dtype, seed=T + 1)


@pytest.mark.parametrize("fmt,n_out", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,k", [(1, 2), (9, 3), (200, 3)])
@pytest.mark.parametrize("blocks", [None, 1, 2, 4, 8, 16])
def test_gated(fmt, n_out, dtype, T, k, blocks, tune):
    if blocks:
        tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    for N, K in ((2, 64), (66, 256), (250, 640)):
        ex = Experts(fmt, 4, N, K, n_out, seed=N)
        check(ex, T, k, dtype, swiglu=True, seed=T)
        check(ex, T, k, dtype, out=dtype, swiglu=True, seed=T)


@pytest.mark.parametrize("fmt,n_out", FORMATS)
@pytest.mark.parametrize("T,k", [(3, 2), (150, 2)])
def test_grouped_input_and_other_output_types(fmt, n_out, T, k):
    ex = Experts(fmt, 4, 72, 256, n_out, seed=3)
    check(ex, T, k, "f16", out="bf16", seed=1, grouped=True)
    check(ex, T, k, "bf16", out="f16", seed=2, grouped=True)


@pytest.mark.parametrize("blocks", [1, 2, 4, 8, 16])
def test_long_rows_and_many_anchors(blocks, tune):
    """K of several windows of group sums, and 3.5% anchors."""
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    for fmt, n_out in (("2bit", 179), ("int4", 51), ("nf4", 0)):
        ex = Experts(fmt, 2, 48, 5120, n_out, seed=9)
        check(ex, 6, 1, "f16", seed=1)
        check(ex, 100, 1, "bf16", seed=2)


def test_all_rows_one_expert_and_none():
    import torch
    ex = Experts("2bit", 6, 80, 256, 0, seed=4)
    rng = np.random.default_rng(1)
    for n in (1, 16, 17, 400):
        for e in (0, 5, -1):
            g, off, rows = device_groups(np.full(n, e), 6)
            x = acts(rng, n, 256, torch.float16)
            Y = torch.full((n, 80), 3.0, device="cuda")
            qw.qgemm_experts(ex.ew, x, g, out=Y)
            if e < 0:
                assert bool((Y == 3.0).all())
                continue
            y, tol = products(ex, x.double().cpu().numpy()[rows], off, is_wide(n, 6), torch.float16)
            assert_close(Y, y, tol, torch.float32)


@pytest.mark.parametrize("blocks", [1, 2, 4, 8, 16])
def test_infinite_and_nan_rows_stay_in_their_rows(blocks, tune):
    """A row's infinities and NaN reach no other row, and none of an anchor
    channel's reach the columns' coded part."""
    import torch
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    for fmt, n_out in FORMATS:
        ex = Experts(fmt, 2, 96, 256, n_out, seed=6)
        for n in (7, 150):
            rng = np.random.default_rng(n)
            ids = rng.integers(0, 2, n).astype(np.int32)
            g, off, rows = device_groups(ids, 2)
            x = acts(rng, n, 256, torch.bfloat16)
            bad = rows[[1, n // 2]]
            clean = qw.qgemm_experts(ex.ew, x, g, out_dtype=torch.float32)
            x[int(bad[0]), 70] = torch.inf
            x[int(bad[1])] = torch.nan
            Y = qw.qgemm_experts(ex.ew, x, g, out_dtype=torch.float32)
            keep = torch.tensor([r not in bad for r in rows], device="cuda")
            assert torch.equal(Y[keep], clean[keep])
            assert not bool(torch.isfinite(Y[n // 2]).any())


@pytest.mark.parametrize("blocks", [1, 2, 4, 8, 16])
def test_offsets_that_do_not_fit_stay_in_bounds(blocks, tune):
    """Offsets beyond the rows, descending or negative, and rows out of range:
    the rows that can be are computed, nothing else is touched."""
    import torch
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    ex = Experts("nf4", 3, 40, 128, 0, seed=8)
    n = 20
    x = acts(np.random.default_rng(0), n, 128, torch.bfloat16)
    for off in ([0, 5, 400, 500], [-7, 3, 2, 20], [0, 0, 0, 0], [20, 20, 20, 20], [0, 20, 0, 20], [9, 0, 20, 1]):
        rows = np.arange(n, dtype=np.int32)
        rows[4] = 10**6
        rows[5] = -3
        g = qw.RowGroups(to_dev(np.array(off, np.int32)), to_dev(rows))
        guard = torch.full((n + 64, 40), 5.0, dtype=torch.bfloat16, device="cuda")
        qw.qgemm_experts(ex.ew, x, g, out=guard[:n])
        torch.cuda.synchronize()
        assert bool((guard[n:] == 5.0).all())


@pytest.mark.parametrize("fmt,n_out", FORMATS)
@pytest.mark.parametrize("T,k,N", [(1, 1, 64), (5, 3, 100), (17, 4, 257), (200, 2, 72)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_combine(fmt, n_out, T, k, N, dtype):
    import torch
    E, K, dt = 4, 320, tdt(dtype)
    ex = Experts(fmt, E, N, K, n_out, seed=N)
    rng = np.random.default_rng(T)
    ids = ids_of(rng, T, k, E, 0.2)
    ids[rng.random((T, k)) < 0.1] = -1  # single empty slots too
    w = rng.random((T, k)).astype(np.float32)
    w[ids < 0] = np.nan  # what an empty slot holds does not matter
    g, off, rows = device_groups(ids, E)
    h = acts(rng, T * k, K, dt)
    y, tol = products(ex, h.double().cpu().numpy(), off, is_wide(T * k, E), dt, is_tall(T * k, ex, dt, torch.float32, False))
    slot_y, slot_t = np.zeros((T * k, N)), np.zeros((T * k, N))
    slot_y[rows[: off[-1]]] = y[: off[-1]]
    slot_t[rows[: off[-1]]] = tol[: off[-1]]
    wz = np.where(ids < 0, 0.0, w).astype(np.float64)[..., None]
    want = (slot_y.reshape(T, k, N) * wz).sum(1)
    lim = ((slot_t.reshape(T, k, N) + k * F32 * np.abs(slot_y.reshape(T, k, N))) * wz).sum(1)
    for out in ("f32", dtype):
        ws = torch.full((qw.qw_experts_combine_workspace_bytes(N, T, k),), 255, dtype=torch.uint8, device="cuda")  # NaN
        got = qw.qgemm_experts_combine(ex.ew, h, g, to_dev(ids), to_dev(w), out_dtype=tdt(out), workspace=ws)
        assert_close(got, want, lim, tdt(out))
        assert bool((got[torch.tensor((ids < 0).all(1), device="cuda")] == 0).all())


def test_one_expert_equals_the_single_matrix_calls():
    """One group of all rows is the product qgemv_* and qgemm_prefill compute."""
    import torch
    rng = np.random.default_rng(2)
    for fmt, n_out in FORMATS:
        ex = Experts(fmt, 1, 96, 512, n_out, seed=12)
        p = ex.packed[0]
        x = acts(rng, 5, 512, torch.float16)
        g, *_ = device_groups(np.zeros(5), 1)
        one = {"2bit": qw.qgemv_2bit, "nf4": qw.qgemv_nf4, "int4": qw.qgemv_int4}[fmt](p, x, out_dtype=torch.float32)
        y = qw.qgemm_experts(ex.ew, x, g, out_dtype=torch.float32)
        assert float((y - one).abs().max()) <= 1e-4 * float(one.abs().max())
        xb = acts(rng, 200, 512, torch.bfloat16)
        g, *_ = device_groups(np.zeros(200), 1)
        pre = qw.qgemm_prefill(p, xb, out_dtype=torch.float32)
        y = qw.qgemm_experts(ex.ew, xb, g, out_dtype=torch.float32)
        assert float((y - pre).abs().max()) <= 1e-2 * float(pre.abs().max())


@pytest.mark.parametrize("blocks", [None, 1, 2, 4])
def test_offsets_beyond_32_bits(blocks, tune):
    """X of more than 4 GiB: rows near its end, by every kernel that takes it."""
    import torch
    if blocks:
        tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    ex = Experts("int4", 2, 48, 8192, 0, seed=21)
    n = 270000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn(n, 8192, generator=gen, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, 2, (n,), generator=gen, device="cuda").to(torch.int32)
    g = qw.qw_group_rows(ids, 2)
    Y = qw.qgemm_experts(ex.ew, x, g, out_dtype=torch.float32)
    rows = g.rows.long()
    off = g.offsets.cpu().numpy()
    for e in range(2):
        at = np.r_[off[e]:off[e] + 3, off[e + 1] - 40:off[e + 1]]
        few = x[rows[torch.from_numpy(at).cuda()]].double().cpu().numpy()
        y, tol = products(ex, few, np.array([0, len(at), len(at)] if e == 0 else [0, 0, len(at)]), True, torch.bfloat16)
        assert_close(Y[torch.from_numpy(at).cuda()], y, tol, torch.float32)


def test_experts_beyond_32_bits():
    """Packed weights of more than 4 GiB: the last experts'."""
    import torch
    E, N, K = 150, 8192, 8192
    codes = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.rand(E, N, K // 64, device="cuda") + 0.5
    ew = qw.ExpertWeights(qw.QW_FMT_NF4_B64, E, N, K, 0, codes, scales)
    level = torch.from_numpy(qw.qw_nf4_levels()).double().cuda()
    for n in (5, 40, 400):
        x = (torch.randn(n, K, device="cuda") / 64).to(torch.bfloat16)
        ids = torch.full((n,), E - 1, dtype=torch.int32, device="cuda")
        ids[::3] = E - 2
        g = qw.qw_group_rows(ids, E)
        Y = qw.qgemm_experts(ew, x, g, out_dtype=torch.float32)
        for e in (E - 1, E - 2):
            q = torch.stack([codes[e] & 15, codes[e] >> 4], -1).flatten(1).long()
            w = level[q] * scales[e].double().repeat_interleave(64, 1)
            at = (ids[g.rows.long()] == e).nonzero()[:, 0]
            xe = x[g.rows.long()[at]].double()
            want, mag = xe @ w.t(), xe.abs() @ w.abs().t()
            # K additions, the levels' (or weights') rounding to bf16
            assert bool(((Y[at].double() - want).abs() <= (K * F32 + 2.0**-8 + F32) * mag).all())


def test_combine_of_most_tokens():
    """More tokens than one launch has workgroups for: all of them."""
    import torch
    E, N, K, T = 2, 8, 64, qw.QW_MAX_ROWS
    codes = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.rand(E, N, K // 64, device="cuda") + 0.5
    ew = qw.ExpertWeights(qw.QW_FMT_NF4_B64, E, N, K, 0, codes, scales)
    level = torch.from_numpy(qw.qw_nf4_levels()).double().cuda()
    ids = torch.randint(0, E, (T, 1), device="cuda", dtype=torch.int32)
    weights = torch.rand(T, 1, device="cuda")
    g = qw.qw_group_rows(ids.flatten(), E)
    h = torch.randn(T, K, device="cuda", dtype=torch.bfloat16)  # grouped order
    out = torch.full((T, N), 7.0, device="cuda")
    qw.qgemm_experts_combine(ew, h, g, ids, weights, out=out)
    at = torch.cat([torch.arange(1000), torch.randint(0, T, (20000,)), torch.arange(T - 1000, T)]).cuda()  # positions
    t = g.rows[at].long()
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(2).long()
    w = level[q] * scales.double()  # (E, N, K): one scale a row
    we, x = w[ids[t, 0].long()], h[at].double()
    want = (we * x[:, None]).sum(-1) * weights[t].double()
    mag = (we * x[:, None]).abs().sum(-1) * weights[t].double()
    # K additions and the weighting, the levels' (or weights') rounding to bf16
    assert bool(((out[t].double() - want).abs() <= (K * F32 + 2.0**-8 + 3 * F32) * mag).all())
    assert int((out == 7.0).all(1).sum()) == 0
