"""GPU: the adapters of many requests added to a shared projection, against
64 bits, elementwise. The inner values t = A x carry K fp32 additions and
two 16-bit parts; out = base + s B t carries theirs through |B|."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import F32, assert_close, device_groups, half_step, tdt

pytestmark = pytest.mark.gpu


def make(n, count, K, N, r, dtype, seed, none=0.2, run=1):
    import torch
    rng = np.random.default_rng(seed)
    dt = tdt(dtype)
    f = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32))
    A, B = (f(count, r, K) / K**0.5).to(dt), (f(count, N, r) / r**0.5).to(dt)
    ad = qw.Adapters(A, B, to_dev(rng.uniform(-2, 2, count).astype(np.float32)))
    ids = np.repeat(rng.integers(0, count, -(-n // run)), run)[:n].astype(np.int32)
    ids[rng.random(n) < none] = -1
    return ad, f(n, K).to(dt), f(n, N), ids


def reference(ad, x, base, ids):
    """Values and bounds in 64 bits."""
    want = base.double().cpu().numpy().copy()
    tol = np.zeros_like(want)
    x = x.double().cpu().numpy()
    two = half_step(ad.dtype) ** 2  # two 16-bit parts
    for a in range(ad.count):
        m = np.flatnonzero(ids == a)
        if not len(m):
            continue
        A, B = ad.A[a].double().cpu().numpy(), ad.B[a].double().cpu().numpy()
        s = float(ad.scale[a])
        t = x[m] @ A.T
        # fp16's second part ends at 2^-24 of the row's largest value
        dt = (ad.K + 64) * F32 * (np.abs(x[m]) @ np.abs(A).T) + two * np.abs(t) + F32 * np.abs(t).max(1, keepdims=True)
        d = s * (t @ B.T)
        want[m] += d
        tol[m] = abs(s) * ((dt + (ad.r + 8) * F32 * np.abs(t)) @ np.abs(B).T) + 2 * F32 * np.abs(d)
    return want, tol


def check(n, count, K, N, r, dtype, seed=0, bases=("f32",), **kw):
    import torch
    ad, x, base32, ids = make(n, count, K, N, r, dtype, seed, **kw)
    g, off, rows = device_groups(ids, count)
    for bdt in bases:
        base = base32.to(tdt(bdt))
        want, tol = reference(ad, x, base, ids)
        tol += F32 * np.abs(want)
        for odt in sorted({"f32", dtype}):
            ws = torch.full((qw.qw_lora_workspace_bytes(ad, n),), 255, dtype=torch.uint8, device="cuda")  # NaN
            out = qw.qw_lora_add(ad, x, g, base, out_dtype=tdt(odt), workspace=ws)
            assert_close(out, want, tol, tdt(odt), f"n={n} K={K} N={N} r={r} {bdt}->{odt}")
            none = torch.tensor(ids < 0, device="cuda")
            assert torch.equal(out[none], base[none].to(tdt(odt)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128, 256])
@pytest.mark.parametrize("n,count", [(1, 1), (1, 7), (5, 3), (64, 32), (100, 2)])
def test_ranks(n, count, r, dtype):
    check(n, count, 320, 200, r, dtype, seed=r + n)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("K,N", [(8, 1), (64, 8), (72, 63), (136, 64), (248, 255), (512, 264), (4096, 1000), (1000, 4097)])
def test_shapes(K, N, dtype):
    for n, count in ((1, 2), (13, 4), (130, 3)):
        check(n, count, K, N, 16, dtype, seed=K + n, bases=("f32", dtype))


@pytest.mark.parametrize("n,count,run", [(1000, 4, 130), (777, 40, 1), (2100, 1, 2100), (300, 200, 1)])
def test_many_rows(n, count, run):
    check(n, count, 512, 520, 32, "bf16", seed=n, run=run, bases=("bf16",))


def test_no_row_has_an_adapter():
    check(9, 3, 128, 100, 8, "f16", none=2.0, bases=("f32", "f16"))
    check(300, 3, 128, 100, 8, "f16", none=2.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n", [6, 200])
def test_in_place(n, dtype):
    import torch
    ad, x, base, ids = make(n, 4, 256, 136, 16, "bf16" if dtype == "f32" else dtype, 3)
    g, *_ = device_groups(ids, 4)
    base = base.to(tdt(dtype))
    want = qw.qw_lora_add(ad, x, g, base)
    got = qw.qw_lora_add(ad, x, g, base, out=base)
    assert got is base and torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0**-13, 2.0**-8, 2.0**7])
def test_inner_values_beyond_16_bits(size, dtype):
    """t far above fp16's largest and far below its smallest normal value,
    by B of the inverse size: the power of two per row keeps the result."""
    import torch
    n, count, K, N, r = 20, 2, 512, 100, 16
    ad, x, base, ids = make(n, count, K, N, r, dtype, 5, none=0)
    A, B = (ad.A.float() * size).to(ad.dtype), (ad.B.float() / size).to(ad.dtype)
    x = (x.float() * size * 8).to(x.dtype)
    ad = qw.Adapters(A, B, ad.scale)
    g, *_ = device_groups(ids, count)
    want, tol = reference(ad, x, base, ids)
    tol += F32 * np.abs(want)
    assert_close(qw.qw_lora_add(ad, x, g, base), want, tol, torch.float32)


def test_zero_and_nonfinite_rows_stay_in_their_rows():
    import torch
    n = 40
    ad, x, base, ids = make(n, 2, 256, 72, 16, "f16", 7, none=0)
    g, *_ = device_groups(ids, 2)
    clean = qw.qw_lora_add(ad, x, g, base)
    x[3, 5], x[8] = torch.inf, torch.nan
    x[11] = 0.0
    out = qw.qw_lora_add(ad, x, g, base)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[3, 8, 11]] = False
    assert torch.equal(out[keep], clean[keep])
    assert torch.equal(out[11], base[11])
    assert bool(torch.isnan(out[8]).all()) and not bool(torch.isfinite(out[3]).any())


def test_offsets_beyond_32_bits():
    """base of more than 4 GiB: its last rows, with and without an adapter."""
    import torch
    n, count, K, N, r = 36000, 3, 64, 32768, 8
    ad, x, _, ids = make(n, count, K, 8, r, "f16", 31, none=0.1)
    B = torch.randn(count, N, r, device="cuda").half()
    ad = qw.Adapters(ad.A, B, ad.scale)
    base = torch.randn(n, N, device="cuda")
    g, *_ = device_groups(ids, count)
    out = qw.qw_lora_add(ad, x, g, base, out_dtype=torch.float16)
    for s in (slice(0, 20), slice(n - 40, n)):
        want, tol = reference(ad, x[s], base[s], ids[s])
        assert_close(out[s], want, tol + F32 * np.abs(want), torch.float16)
