"""The calls around a projection run together, as a decoder layer would: norm,
projections with bias, activation, gate and residual, router, experts. Every
stage is held against the formula in 64 bits of what the stage before it wrote;
the chain gives the same bits on another stream and replayed from a graph; calls
beyond 32-bit offsets agree with small ones."""

import numpy as np
import pytest

from bit_weight_quantized_qw_amd import qw
from layer_util import Matrix, TOP, linear64, xdt
from routed_util import F32, Experts, assert_close, tdt

pytestmark = pytest.mark.gpu

H, I, E, K_TOP = 512, 768, 16, 4


class Layer:
    def __init__(self, seed=0):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.o = Matrix("nf4", H, H, 0, seed)
        self.gu = Matrix("int4", 2 * I, H, 5, seed + 1)
        self.down = Matrix("2bit", H, I, 27, seed + 2)
        self.router = Matrix("nf4", E, H, 0, seed + 3)
        self.experts = Experts("2bit", E, 2 * 64, H, 0, seed + 4)
        self.back = Experts("nf4", E, H, 64, 0, seed + 5)
        self.g1 = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
        self.g2 = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().cuda()
        self.bias = (0.1 * torch.randn(H, generator=g)).cuda()
        self.balance = (0.05 * torch.randn(E, generator=g)).cuda()

    def run(self, x, stream):
        """x (M, H) bf16: what attention left; stream (M, H) fp32: the residual."""
        import torch
        s = {"o": qw.qgemm_linear(self.o.pw, x, bias=self.bias, residual=stream, out_dtype=torch.float32)}
        s["n1"] = qw.qw_rmsnorm(s["o"], self.g1, out_dtype=torch.float8_e4m3fn)
        s["mid"] = qw.qgemm_linear(self.gu.pw, s["n1"].y, x_scales=s["n1"].scales, act="silu", gated=True, out_dtype=torch.bfloat16)
        s["ffn"] = qw.qgemm_linear(self.down.pw, s["mid"])
        s["n2"] = qw.qw_rmsnorm(s["ffn"], self.g2, residual=s["o"], out_dtype=torch.bfloat16)
        s["logits"] = qw.qgemm_linear(self.router.pw, s["n2"].y, out_dtype=torch.float32)
        r = s["route"] = qw.qw_route_scored(s["logits"], K_TOP, bias=self.balance, n_groups=4, top_groups=2, scale=2.5)
        mid = qw.qgemm_experts(self.experts.ew, s["n2"].y, r.groups, top_k=K_TOP, swiglu=True)
        s["y"] = qw.qgemm_experts_combine(self.back.ew, mid, r.groups, r.ids, r.weights)
        return s


def flat(s):
    out = []
    for v in s.values():
        out += [t for t in ([v.y, v.scales, v.residual] if isinstance(v, qw.Normed) else
                            [v.ids, v.weights, v.groups.offsets, v.groups.rows] if isinstance(v, qw.Routing) else [v]) if t is not None]
    return out


def same(a, b):
    import torch
    return all(torch.equal(u.view(torch.uint8) if u.dtype == torch.float8_e4m3fn else u,
                           v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v) for u, v in zip(flat(a), flat(b)))


def start(M, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn(M, H, generator=g).bfloat16().cuda(), (3 * torch.randn(M, H, generator=g)).cuda()


@pytest.mark.parametrize("M", [1, 6, 50, 300])
def test_every_stage_against_its_input(M):
    layer = Layer()
    x, stream = start(M, M)
    s = layer.run(x, stream)
    d = lambda t: t.double().cpu().numpy()
    v, tol = linear64(layer.o, d(x), "bf16", M > 32, d(layer.bias), residual=d(stream))
    assert_close(s["o"], v, tol, tdt("f32"), "o")
    o = d(s["o"])
    n = o / np.sqrt((o * o).mean(1, keepdims=True) + 1e-6) * d(layer.g1)
    scale = d(s["n1"].scales)
    rel = (H / 2 + 16) * F32
    assert (np.abs(scale - np.abs(n).max(1) / TOP["e4m3"]) <= rel * scale).all()
    q = s["n1"].y.float().double().cpu().numpy()
    want = n / scale[:, None]
    assert (np.abs(q - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2 * rel * np.abs(want)).all()
    v, tol = linear64(layer.gu, q * scale[:, None], "e4m3", M > 32, act="silu", gated=True)
    assert_close(s["mid"], v, tol, tdt("bf16"), "mid")
    v, tol = linear64(layer.down, d(s["mid"]), "bf16", M > 32)
    assert_close(s["ffn"], v, tol, tdt("bf16"), "ffn")
    h = d(s["ffn"]) + o
    assert_close(s["n2"].residual, h, F32 * np.abs(h), tdt("f32"), "residual")
    n = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * d(layer.g2)
    assert_close(s["n2"].y, n, rel * np.abs(n), tdt("bf16"), "n2")
    v, tol = linear64(layer.router, d(s["n2"].y), "bf16", M > 32)
    assert_close(s["logits"], v, tol, tdt("f32"), "logits")
    from test_gpu_route_scored import oracle
    ids, w = oracle(d(s["logits"]), K_TOP, "sigmoid", layer.balance.cpu().numpy(), 4, 2, "top2", True, 2.5)
    assert np.array_equal(s["route"].ids.cpu().numpy(), ids)
    assert (np.abs(d(s["route"].weights) - w) <= (F32 + 1e-12) * w).all()
    # the experts on the routed rows, each token's sum
    X = d(s["n2"].y)
    y = np.zeros((M, H))
    for t in range(M):
        for j, e in enumerate(ids[t]):
            z = layer.experts.W[e] @ X[t]
            gate, up = z[:64], z[64:]
            mid = (gate / (1 + np.exp(-gate)) * up)
            y[t] += w[t, j] * (layer.back.W[e] @ mid)
    # two products with bf16 between them: 2^-8 of a term, at most, is a bound on the norm
    assert np.abs(d(s["y"]) - y).max() <= 2.0 ** -7 * np.abs(y).max()


def test_other_streams_and_replays():
    """On a side stream beside other work, and captured: three replays with new
    inputs, eager calls between them, all equal to eager runs."""
    import torch
    layer = Layer(20)
    for M in (5, 120):
        x, stream = start(M, 1)
        want = layer.run(x, stream)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = [layer.run(x, stream) for _ in range(3)]
        beside = [layer.run(x, stream) for _ in range(3)]  # at the same time, on the default stream
        side.synchronize()
        torch.cuda.synchronize()
        assert all(same(want, g) for g in got + beside)
        sx, ss = x.clone(), stream.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.run(sx, ss)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer.run(sx, ss)
        for seed in (2, 3, 4):
            nx, ns = start(M, seed)
            sx.copy_(nx)
            ss.copy_(ns)
            graph.replay()
            eager = layer.run(nx, ns)
            torch.cuda.synchronize()
            assert same(out, eager), (M, seed)


def test_the_same_bits_every_time():
    layer = Layer(30)
    for M in (3, 40, 400):
        x, stream = start(M, 7)
        a = layer.run(x, stream)
        assert all(same(a, layer.run(x, stream)) for _ in range(3))


def test_kernel_times_are_recorded():
    import torch
    layer = Layer(31)
    x, stream = start(200, 8)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    logits = torch.randn(200, E, device="cuda")
    for call in (lambda: qw.qgemm_linear(layer.o.pw, x, residual=stream), lambda: qw.qw_rmsnorm(x, layer.g1),
                 lambda: qw.qw_route_scored(logits, 4)):
        qw.qw_time_next_call(a, b)
        call()
        torch.cuda.synchronize()
        assert 0 < a.elapsed_time(b) < 1000


def test_given_workspaces(tune):
    import torch
    layer = Layer(32)
    tune(qw.QW_TUNE_LINEAR_PARTS, 2)
    x, _ = start(100, 9)
    nb = qw.qw_linear_workspace_bytes(layer.o.pw, x.dtype, 100)
    assert nb == 2 * 100 * H * 4
    want = qw.qgemm_linear(layer.o.pw, x)
    ws = torch.full((nb + 64,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(qw.qgemm_linear(layer.o.pw, x, workspace=ws), want) and bool((ws[nb:] == 255).all())
    with pytest.raises(ValueError):
        qw.qgemm_linear(layer.o.pw, x, workspace=ws[: nb - 1])
    logits = torch.randn(3000, E, device="cuda")
    nb = qw.qw_route_scored_workspace_bytes(3000, E, 4, 2)
    assert nb > 0
    with pytest.raises(ValueError):
        qw.qw_route_scored(logits, 4, n_groups=2, workspace=torch.empty(nb - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("blocks", [1, 2, 8, 16])
def test_activations_beyond_2_gib(tune, blocks):
    """X of 2.1 GiB: the last rows are those of a small call."""
    import torch
    tune(qw.QW_TUNE_LINEAR_ROW_BLOCKS, blocks)
    tune(qw.QW_TUNE_LINEAR_PARTS, 1)
    K, M = 4096, 282000
    m = Matrix("int4", 24, K, 3, 40)
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.float16)
    r = torch.randn(M, 24, generator=g, device="cuda")
    y = qw.qgemm_linear(m.pw, X, residual=r)
    for at in (0, 131072, 262016, M - 128):  # tiles' first rows
        part = qw.qgemm_linear(m.pw, X[at:at + 128], residual=r[at:at + 128])
        assert torch.equal(y[at:at + 128], part), at


def test_outputs_beyond_2_gib():
    import torch
    m = Matrix("int4", 4100, 64, 0, 41)
    M = 140000
    X = torch.randn(M, 64, device="cuda", dtype=torch.bfloat16)
    y = qw.qgemm_linear(m.pw, X, act="relu", out_dtype=torch.float32)
    for at in (0, 130944, M - 128):
        want, tol = linear64(m, X[at:at + 128].double().cpu().numpy(), "bf16", True, act="relu")
        assert_close(y[at:at + 128], want, tol, tdt("f32"), f"rows {at}")


@pytest.mark.parametrize("y", ["f16", "i8"])
def test_norms_beyond_2_gib(y):
    import torch
    M, K = 70000, 16384
    x = torch.randn(M, K, device="cuda", dtype=torch.float16)
    w = torch.randn(K, device="cuda", dtype=torch.float16)
    n = qw.qw_rmsnorm(x, w, residual=x, out_dtype=xdt(y))
    part = qw.qw_rmsnorm(x[-9:], w, residual=x[-9:], out_dtype=xdt(y))
    assert torch.equal(n.y[-9:], part.y) and torch.equal(n.residual[-9:], part.residual)
    assert n.scales is None or torch.equal(n.scales[-9:], part.scales)


def test_many_tokens_routed():
    import torch
    T = 400000
    logits = torch.randn(T, 64, device="cuda", dtype=torch.bfloat16)
    bias = 0.1 * torch.randn(64, device="cuda")
    r = qw.qw_route_scored(logits, 6, bias=bias, n_groups=8, top_groups=3)
    part = qw.qw_route_scored(logits[-1000:], 6, bias=bias, n_groups=8, top_groups=3)
    assert torch.equal(r.ids[-1000:], part.ids) and torch.equal(r.weights[-1000:], part.weights)
    g = qw.qw_group_rows(r.ids.view(-1), 64)
    assert torch.equal(g.offsets, r.groups.offsets) and torch.equal(g.rows, r.groups.rows)
