"""GPU: offsets and rows that do not fit, in memory that does. Offsets are
clamped to 0..n, a descending pair is an empty group, rows out of range are
skipped: the rows that remain are computed, and everything else stays as it
was, in front of the output, in it and behind it."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import F32, Experts, assert_close, half_step

pytestmark = pytest.mark.gpu

G, LEFT = 3, 5.0  # groups; what memory holds that no call may write
GUARD = 64        # rows in front of and behind an output


def offsets(n):
    """Offsets that do not fit n rows; some let two groups overlap."""
    return [[0, n // 4, 20 * n, 25 * n], [-7, n // 6, n // 8, n], [0, 0, 0, 0], [n, n, n, n], [n // 2, 0, n, 1],
            [n // 3, n // 2, n // 2 + 1, n - 2], [0, -2**31, 2**31 - 1, 2**31 - 1]]


def covering(off, n):
    """For every position the groups that hold it, from the clamped offsets."""
    at = [[] for _ in range(n)]
    for g in range(G):
        lo = min(max(off[g], 0), n)
        for p in range(lo, min(max(off[g + 1], lo), n)):
            at[p].append(g)
    return at


def bad_rows(n, rng):
    """A permutation with entries replaced by others out of range."""
    rows = rng.permutation(n).astype(np.int32)
    at = rng.choice(n, 8, replace=False)
    rows[at] = [10**6, -1, -2, -3, -n, 2**31 - 1, -2**31, 3 * n]
    return rows


def guarded(n, cols, dtype):
    import torch
    t = torch.full((n + 2 * GUARD, cols), LEFT, dtype=dtype, device="cuda")
    return t, t[GUARD:GUARD + n]


def check_rows(whole, out, want, tol, at, what):
    """Row p of out is the groups' at[p] (want[g][p]; of two groups that hold
    it, the later store of each element), or as it was."""
    import torch
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    lim = [tol[g] + half_step(out.dtype) * (np.abs(want[g]) + tol[g]) for g in range(len(want))]
    for p, groups in enumerate(at):
        if groups:
            ok = np.stack([np.abs(got[p] - want[g][p]) <= lim[g][p] for g in groups])
            assert ok.any(0).all(), f"{what}: row {p}"
        else:
            assert (got[p] == LEFT).all(), f"{what}: row {p} was written"
    assert bool((whole[:GUARD] == LEFT).all() and (whole[-GUARD:] == LEFT).all()), f"{what}: written beside the output"


def rounding(ex, dtype):
    """Share of the terms that any of the kernels may round away: the widest."""
    return half_step(dtype) + F32


@pytest.mark.parametrize("blocks", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("fmt", ["nf4", "2bit", "int4"])
@pytest.mark.parametrize("n", [20, 400])
@pytest.mark.parametrize("top_k", [None, 1, 2, 3])
def test_experts(blocks, fmt, n, top_k, tune):
    import torch
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    N, K, dt = 72, 128, torch.bfloat16
    ex = Experts(fmt, G, N, K, 0, seed=3)
    rng = np.random.default_rng(n)
    x_rows = n if top_k is None else -(-n // top_k)
    x = to_dev(rng.standard_normal((x_rows, K)).astype(np.float32)).to(dt)
    x64 = x.double().cpu().numpy()
    for off in offsets(n):
        rows = bad_rows(n, rng)
        whole, out = guarded(n, N, dt)
        g = qw.RowGroups(to_dev(np.array(off, np.int32)), to_dev(rows))
        qw.qgemm_experts(ex.ew, x, g, top_k=top_k, out=out)
        at = covering(off, n)
        r = np.arange(n)
        if top_k is not None:
            r = np.where(rows < 0, -1, rows.astype(np.int64) // top_k)
            at = [a if 0 <= r[p] < x_rows else [] for p, a in enumerate(at)]
        xr = x64[np.clip(r, 0, x_rows - 1)]
        want = [xr @ ex.W[e].T for e in range(G)]
        tol = [((K + 64) * F32 + rounding(ex, dt)) * (np.abs(xr) @ ex.mag[e].T) for e in range(G)]
        check_rows(whole, out, want, tol, at, f"{fmt} {off}")


@pytest.mark.parametrize("blocks", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("T", [10, 200])
def test_combine(blocks, T, tune):
    """Slots that no position stores keep what the workspace held: 0 here."""
    import torch
    tune(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, blocks)
    k, N, K, dt = 2, 72, 128, torch.bfloat16
    n = T * k
    ex = Experts("nf4", G, N, K, 0, seed=4)
    rng = np.random.default_rng(T)
    h = to_dev(rng.standard_normal((n, K)).astype(np.float32)).to(dt)
    h64 = h.double().cpu().numpy()
    w = rng.random((T, k)).astype(np.float32)
    ids = rng.integers(-1, G, (T, k)).astype(np.int32)
    for off in offsets(n):
        at = covering(off, n)
        if max(len(a) for a in at) > 1:  # which group's product a slot keeps is open
            continue
        rows = bad_rows(n, rng)
        whole, out = guarded(T, N, dt)
        need = qw.qw_experts_combine_workspace_bytes(N, T, k)
        ws = torch.zeros(need + 8192, dtype=torch.uint8, device="cuda")
        ws[:4096] = ws[-4096:] = 85
        g = qw.RowGroups(to_dev(np.array(off, np.int32)), to_dev(rows))
        qw.qgemm_experts_combine(ex.ew, h, g, to_dev(ids), to_dev(w), out=out, workspace=ws[4096:4096 + need])
        torch.cuda.synchronize()
        assert bool((ws[:4096] == 85).all() and (ws[-4096:] == 85).all())
        P, tol = np.zeros((n, N)), np.zeros((n, N))
        for p, a in enumerate(at):
            if a and 0 <= rows[p] < n:
                P[rows[p]] = h64[p] @ ex.W[a[0]].T
                tol[rows[p]] = ((K + 64) * F32 + rounding(ex, dt)) * (np.abs(h64[p]) @ ex.mag[a[0]].T)
        wz = np.where(ids < 0, 0.0, w).astype(np.float64)[..., None]
        want = (P.reshape(T, k, N) * wz).sum(1)
        lim = ((tol + k * F32 * np.abs(P)).reshape(T, k, N) * wz).sum(1)
        check_rows(whole, out, [want], [lim], [[0]] * T, f"combine {off}")


@pytest.mark.parametrize("n", [20, 64, 65, 400])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N", [72, 67])
def test_adapters(n, in_place, N):
    import torch
    K, r, dt = 128, 16, torch.bfloat16
    rng = np.random.default_rng(n)
    f = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32))
    ad = qw.Adapters((f(G, r, K) / 11).to(dt), (f(G, N, r) / 4).to(dt), f(G))
    A, B, s = ad.A.double().cpu().numpy(), ad.B.double().cpu().numpy(), ad.scale.double().cpu().numpy()
    x = f(n, K).to(dt)
    x64 = x.double().cpu().numpy()
    for off in offsets(n):
        at = covering(off, n)
        end = min(max(off[G], 0), n)
        for p in range(end, n):
            at[p].append(G)  # behind the last group: base alone
        if max(len(a) for a in at) > 1:  # in place, two groups' sums
            continue
        rows = bad_rows(n, rng)
        whole, out = guarded(n, N, torch.float32)
        base = f(n, N)
        if in_place:
            out.copy_(base)
        g = qw.RowGroups(to_dev(np.array(off, np.int32)), to_dev(rows))
        qw.qw_lora_add(ad, x, g, out if in_place else base, out=out)
        b64 = base.double().cpu().numpy()
        want, tol = np.full((n, N), LEFT), np.zeros((n, N))
        if in_place:
            want = b64.copy()
        for p, a in enumerate(at):
            m = rows[p]
            if not a or not 0 <= m < n:
                continue
            want[m] = b64[m]
            if a[0] < G:
                t = A[a[0]] @ x64[m]
                dt_ = (K + 64) * F32 * (np.abs(A[a[0]]) @ np.abs(x64[m])) + 2.0**-16 * np.abs(t) + F32 * np.abs(t).max()
                d = s[a[0]] * (B[a[0]] @ t)
                want[m] += d
                tol[m] = abs(s[a[0]]) * (np.abs(B[a[0]]) @ (dt_ + (r + 8) * F32 * np.abs(t))) + 2 * F32 * np.abs(d) + F32 * np.abs(want[m])
        check_rows(whole, out, [want], [tol], [[0]] * n, f"adapters {off}")


@pytest.mark.parametrize("E,n", [(150, 5)])
def test_few_rows_of_experts_beyond_32_bits(E, n):
    """Packed weights of more than 4 GiB: the last experts' products by the
    kernel of few rows, whose bound is that of two-part levels."""
    import torch
    N, K = 8192, 8192
    codes = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.rand(E, N, K // 64, device="cuda") + 0.5
    ew = qw.ExpertWeights(qw.QW_FMT_NF4_B64, E, N, K, 0, codes, scales)
    level = torch.from_numpy(qw.qw_nf4_levels()).double().cuda()
    x = (torch.randn(n, K, device="cuda") / 64).to(torch.bfloat16)
    ids = torch.full((n,), E - 1, dtype=torch.int32, device="cuda")
    ids[::3] = E - 2
    g = qw.qw_group_rows(ids, E)
    with qw.tuned(qw.QW_TUNE_EXPERTS_ROW_BLOCKS, 1):
        Y = qw.qgemm_experts(ew, x, g, out_dtype=torch.float32)
    for e in (E - 1, E - 2):
        q = torch.stack([codes[e] & 15, codes[e] >> 4], -1).flatten(1).long()
        w = level[q] * scales[e].double().repeat_interleave(64, 1)
        at = (ids[g.rows.long()] == e).nonzero()[:, 0]
        xe = x[g.rows.long()[at]].double()
        want, mag = xe @ w.t(), xe.abs() @ w.abs().t()
        assert bool(((Y[at].double() - want).abs() <= ((K + 64) * F32 + 2.0**-16) * mag + F32 * want.abs()).all())
