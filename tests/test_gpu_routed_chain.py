"""GPU: the routed calls as a decoder block uses them: a shared packed
projection with the requests' adapters, a router, the experts' gated
products and their weighted sum. Each stage is checked against 64 bits on
the stage's own inputs; then the chain on another stream, captured and
replayed, in two streams at once, and again for the same bits."""

import numpy as np
import pytest

import oracle
from bit_weight_quantized_qw_amd import qw
from gpu_util import to_dev
from routed_util import F32, Experts, assert_close, gated, group, half_step, products, tdt

pytestmark = pytest.mark.gpu

E, K, I, TOPK, ADAPTERS, RANK = 6, 256, 192, 3, 4, 16


class Block:
    """Weights of one block and its buffers for T tokens."""

    def __init__(self, T, dtype, seed=0):
        import torch
        rng = np.random.default_rng(seed)
        self.T, self.dt = T, tdt(dtype)
        w = (rng.standard_normal((K, K)) * 0.05).astype(np.float32)
        self.proj = qw.qw_pack(to_dev(w), qw.QW_FMT_NF4_B64)
        self.proj64 = oracle.dequant_nf4(oracle.unpack_nf4(self.proj.host_codes()), self.proj.host_scales().astype(np.float64))
        f = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32))
        self.ad = qw.Adapters((f(ADAPTERS, RANK, K) / 16).to(self.dt), (f(ADAPTERS, K, RANK) / 16).to(self.dt), f(ADAPTERS))
        self.router = f(K, E) / 16
        self.up = Experts("int4", E, 2 * I, K, 3, seed=seed + 1)
        self.down = Experts("2bit", E, K, I, 5, seed=seed + 2)
        self.ids = to_dev(rng.integers(-1, ADAPTERS, T).astype(np.int32))
        self.x = f(T, K).to(self.dt)
        ws = lambda n: torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        self.ws = [ws(qw.qw_group_rows_workspace_bytes(T, ADAPTERS)), ws(qw.qw_lora_workspace_bytes(self.ad, T)),
                   ws(qw.qw_route_workspace_bytes(T, E, TOPK)), ws(qw.qw_experts_combine_workspace_bytes(K, T, TOPK))]

    def new_inputs(self, seed):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.x.copy_(torch.randn(self.T, K, generator=g, device="cuda").to(self.dt))
        self.ids.copy_(torch.randint(-1, ADAPTERS, (self.T,), generator=g, device="cuda").to(torch.int32))

    def run(self):
        import torch
        groups = qw.qw_group_rows(self.ids, ADAPTERS, workspace=self.ws[0])
        if self.dt == torch.float16:
            base = torch.cat([qw.qgemv_nf4(self.proj, self.x[i:i + 8], out_dtype=torch.float32) for i in range(0, self.T, 8)])
        else:
            base = qw.qgemm_prefill(self.proj, self.x, out_dtype=torch.float32)
        h = qw.qw_lora_add(self.ad, self.x, groups, base, out_dtype=self.dt, workspace=self.ws[1])
        logits = (h.float()[:, :, None] * self.router).sum(1)
        r = qw.qw_route_topk(logits, TOPK, workspace=self.ws[2])
        mid = qw.qgemm_experts(self.up.ew, h, r.groups, top_k=TOPK, swiglu=True)
        y = qw.qgemm_experts_combine(self.down.ew, mid, r.groups, r.ids, r.weights, workspace=self.ws[3])
        return {"groups": groups, "base": base, "h": h, "logits": logits, "r": r, "mid": mid, "y": y}


def bits(o):
    return [o["base"], o["h"], o["logits"], o["r"].ids, o["r"].weights, o["r"].groups.rows, o["mid"], o["y"]]


@pytest.mark.parametrize("T,dtype", [(1, "f16"), (7, "f16"), (40, "f16"), (33, "bf16"), (900, "bf16")])
def test_stages(T, dtype):
    import torch
    b = Block(T, dtype, seed=T)
    o = b.run()
    x = b.x.double().cpu().numpy()
    # projection and adapters
    ids = b.ids.cpu().numpy()
    off, rows = group(ids, ADAPTERS)
    np.testing.assert_array_equal(o["groups"].rows.cpu().numpy(), rows)
    want = o["base"].double().cpu().numpy().copy()
    tol = 2 * F32 * np.abs(want)
    assert np.abs(want - x @ b.proj64.T).max() <= 4e-3 * np.abs(x @ b.proj64.T).max()
    for a in range(ADAPTERS):
        m = np.flatnonzero(ids == a)
        if len(m):
            A, B, s = b.ad.A[a].double().cpu().numpy(), b.ad.B[a].double().cpu().numpy(), float(b.ad.scale[a])
            t = x[m] @ A.T
            dt = (K + 64) * F32 * (np.abs(x[m]) @ np.abs(A).T) + half_step(b.dt) ** 2 * np.abs(t) + F32 * np.abs(t).max(1, keepdims=True)
            want[m] += s * (t @ B.T)
            tol[m] += abs(s) * ((dt + (RANK + 8) * F32 * np.abs(t)) @ np.abs(B).T) + 2 * F32 * np.abs(want[m])
    assert_close(o["h"], want, tol, b.dt, "adapters")
    # router
    lg = o["logits"].double().cpu().numpy()
    top = np.argsort(-lg, axis=1, kind="stable")[:, :TOPK]
    np.testing.assert_array_equal(o["r"].ids.cpu().numpy(), top)
    roff, rrows = group(top, E)
    np.testing.assert_array_equal(o["r"].groups.rows.cpu().numpy(), rrows)
    # experts: every kernel's bound is within the widest
    h = o["h"].double().cpu().numpy()
    y, tol = gated(*products(b.up, h[rrows // TOPK], roff, True, b.dt))
    assert_close(o["mid"], y, tol, b.dt, "gated")
    mid = o["mid"].double().cpu().numpy()
    y, tol = products(b.down, mid, roff, True, b.dt)
    sy, st = np.zeros_like(y), np.zeros_like(tol)
    sy[rrows], st[rrows] = y, tol
    w = o["r"].weights.double().cpu().numpy()[..., None]
    sy, st = sy.reshape(T, TOPK, K), st.reshape(T, TOPK, K)
    assert_close(o["y"], (sy * w).sum(1), ((st + TOPK * F32 * np.abs(sy)) * w).sum(1), b.dt, "combine")


@pytest.mark.parametrize("T,dtype", [(5, "f16"), (300, "bf16")])
def test_same_bits_again_and_on_another_stream(T, dtype):
    import torch
    b = Block(T, dtype)
    first = bits(b.run())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = bits(b.run())
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for again in (bits(b.run()), other):
        for p, q in zip(first, again):
            assert torch.equal(p, q)


@pytest.mark.parametrize("T,dtype", [(5, "f16"), (300, "bf16")])
def test_graph_replays_equal_eager(T, dtype):
    import torch
    b = Block(T, dtype)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = b.run()
    for seed in range(4):
        b.new_inputs(seed)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in bits(held)]
        want = bits(b.run())
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


def test_two_streams_at_once():
    """Two chains on two streams, each with its own workspaces, interleaved."""
    import torch
    a, b = Block(200, "bf16", seed=1), Block(40, "f16", seed=2)
    want = bits(a.run()), bits(b.run())
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            oa = a.run()
        with torch.cuda.stream(t):
            ob = b.run()
        torch.cuda.synchronize()
        for w, o in zip(want, (oa, ob)):
            for p, q in zip(w, bits(o)):
                assert torch.equal(p, q)


def test_binding_refusals():
    import torch
    b = Block(6, "f16")
    g = qw.qw_group_rows(b.ids, ADAPTERS)
    base = torch.zeros(6, K, device="cuda")
    with pytest.raises(ValueError):
        qw.qw_lora_add(b.ad, b.x[:5], g, base[:5])            # groups of another number of rows
    with pytest.raises(ValueError):
        qw.qw_lora_add(b.ad, b.x, g, base[:, :-1])
    with pytest.raises(TypeError):
        qw.qw_lora_add(b.ad, b.x.bfloat16(), g, base)
    with pytest.raises(ValueError):
        qw.qw_lora_add(b.ad, b.x, g, base.t().contiguous().t())  # not contiguous
    with pytest.raises(TypeError):
        qw.qw_lora_add(b.ad, b.x, g, base.int())
    with pytest.raises(ValueError):
        qw.qw_lora_add(b.ad, b.x, g, base, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    r = qw.qw_route_topk(torch.randn(6, E, device="cuda"), TOPK)
    with pytest.raises(ValueError):
        qw.qgemm_experts(b.up.ew, b.x[:5], r.groups, top_k=TOPK)  # slots of rows that are not there
    with pytest.raises(ValueError):
        qw.qgemm_experts(b.up.ew, b.x, g)                      # groups of another number of experts
    with pytest.raises(ValueError):
        qw.qgemm_experts(b.up.ew, b.x, r.groups, top_k=None)   # grouped order needs a row per slot
    with pytest.raises(TypeError):
        qw.qgemm_experts(b.up.ew, b.x.float(), r.groups, top_k=TOPK)
    with pytest.raises(ValueError):
        qw.qgemm_experts(b.up.ew, b.x, r.groups, top_k=TOPK, out=torch.zeros(18, I, device="cuda"))
    with pytest.raises(ValueError):
        qw.qgemm_experts_combine(b.down.ew, b.x, r.groups, r.ids, r.weights)
    for k in (0, E + 1):
        with pytest.raises(ValueError):
            qw.qw_route_topk(torch.randn(6, E, device="cuda"), k)
    with pytest.raises(qw.QwError) as e:
        qw.qw_route_topk(torch.randn(2, 2000, device="cuda"), 2)
    assert e.value.status == qw.QW_ERR_UNSUPPORTED
