"""The operators around a layer's packed projections, as cases to measure.

Three operators: ``norm`` (the root-mean-square norm with the residual's
addition, its output in 16 bits, in 8 bits with a scale a row, or in the INT4
format's channel order), ``linear`` (the product with a packed matrix, with
bias, activation, gate and residual behind it, of activations in 16 or 8
bits) and ``route`` (a router with softmax or sigmoid scores, a balancing
bias and groups of experts).

``run`` computes a case in its plain form (elementary torch operations) or,
where ``own`` is true, by the library's calls. ``exact`` computes the
definition in 64 bits.
"""

import math
from statistics import NormalDist

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
CODEBOOK = [-1.52, -0.45, 0.45, 1.52]
GROUP = {"2bit": 32, "nf4": 64, "int4": 32}          # weights per scale
ANCHORS = {"2bit": 0.035, "nf4": 0.0, "int4": 0.01}  # share of the channels kept in fp16
TOP = {"e4m3": 448.0, "i8": 127.0}                   # the largest number of an 8-bit type


def _nf4_levels():
    """The 16 NF4 levels: normal quantiles at evenly spaced probabilities,
    eight above zero, seven below, and zero, divided by the largest."""
    n, delta = NormalDist(), 1 - 0.5 * (1 / 32 + 1 / 30)
    v = [n.inv_cdf(delta + (0.5 - delta) * i / 8) for i in range(8)]
    v += [-n.inv_cdf(delta + (0.5 - delta) * i / 7) for i in range(7)] + [0.0]
    return [x / max(v) for x in sorted(v)]


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden state before a layer's projections: latency
        {"name": "norm_token", "op": "norm", "M": 1, "K": 5120, "x": "f16", "residual": "f16", "y": "f16", "perm": False},
        # a short prompt before an INT4 projection: y in its channel order, an fp32 residual stream
        {"name": "norm_permuted", "op": "norm", "M": 777, "K": 5120, "x": "bf16", "residual": "f32", "y": "bf16", "perm": True},
        # a long prompt's tokens, written in 8 bits for the next product
        {"name": "norm_prefill", "op": "norm", "M": 8192, "K": 8192, "x": "bf16", "residual": "bf16", "y": "e4m3", "perm": False},
        # one token's output projection with the residual stream added: latency
        {"name": "linear_token", "op": "linear", "M": 1, "K": 5120, "N": 5120, "fmt": "2bit", "anchors": True, "x": "f16",
         "bias": False, "act": None, "gated": False, "residual": "f16", "y": "f16"},
        # a decode batch between the batches that a GEMV and a prefill are made for
        {"name": "linear_batch", "op": "linear", "M": 24, "K": 4096, "N": 11008, "fmt": "nf4", "anchors": False, "x": "bf16",
         "bias": True, "act": "gelu_tanh", "gated": False, "residual": None, "y": "bf16"},
        # a small decode batch's down projection, from 8-bit activations: the weights' stream
        {"name": "linear_decode", "op": "linear", "M": 7, "K": 28672, "N": 8192, "fmt": "int4", "anchors": True, "x": "e4m3",
         "bias": False, "act": None, "gated": False, "residual": "bf16", "y": "bf16"},
        # a short ragged prompt, an odd number of columns, fp16 anchors, 8-bit activations
        {"name": "linear_ragged", "op": "linear", "M": 333, "K": 2048, "N": 1501, "fmt": "2bit", "anchors": True, "x": "i8",
         "bias": True, "act": "silu", "gated": False, "residual": "f32", "y": "f16"},
        # a prompt's merged gate and up projections
        {"name": "linear_gated", "op": "linear", "M": 2000, "K": 5120, "N": 27648, "fmt": "int4", "anchors": False, "x": "bf16",
         "bias": False, "act": "silu", "gated": True, "residual": None, "y": "bf16"},
        # a long prompt through a large matrix: the matrix cores' rate
        {"name": "linear_prefill", "op": "linear", "M": 2048, "K": 8192, "N": 28672, "fmt": "2bit", "anchors": False, "x": "bf16",
         "bias": True, "act": "relu", "gated": False, "residual": "bf16", "y": "bf16"},
        # a decode batch's router, a tenth of the slots padding
        {"name": "route_decode", "op": "route", "T": 64, "E": 256, "k": 8, "dtype": "f32", "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "by": "top2", "norm": True, "scale": 2.5, "pad": 0.1},
        # fewer experts, softmax scores, groups by their best expert
        {"name": "route_softmax", "op": "route", "T": 1001, "E": 160, "k": 6, "dtype": "bf16", "score": "softmax", "bias": False,
         "groups": 8, "top_groups": 3, "by": "max", "norm": False, "scale": 16.0, "pad": 0.0},
        # the tokens of a prefill
        {"name": "route_prefill", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "f32", "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "by": "top2", "norm": True, "scale": 2.5, "pad": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "linear", "route"])
    if op == "norm":
        c = {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 100, 8192), "x": rng.choice(["f16", "bf16"]),
             "residual": rng.choice([None, "f16", "bf16", "f32"]), "y": rng.choice(["f16", "bf16", "e4m3", "i8"]),
             "perm": rng.random() < 0.3}
        if rng.random() < 0.6:  # most models' widths are multiples of 64
            c["K"] = max(128, c["K"] // 64 * 64)
        return c
    if op == "route":
        E, groups = rng.choice([(16, 1), (60, 4), (64, 8), (100, 5), (128, 4), (160, 8), (256, 8), (384, 1)])
        top_groups = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E // groups * top_groups)),
                "dtype": rng.choice(["f32", "bf16", "f16"]), "score": rng.choice(["sigmoid", "softmax"]), "bias": rng.random() < 0.6,
                "groups": groups, "top_groups": top_groups, "by": rng.choice(["max", "top2"]), "norm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "pad": rng.choice([0.0, 0.1])}
    fmt, x = rng.choice(["2bit", "nf4", "int4"]), rng.choice(["f16", "bf16", "e4m3", "i8"])
    y = rng.choice(["f16", "bf16"])
    c = {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 512, 28672, 64), "N": _log(rng, 500, 28672), "fmt": fmt,
         "anchors": fmt != "nf4" and rng.random() < 0.4, "x": x, "bias": rng.random() < 0.5,
         "act": rng.choice([None, "relu", "silu", "gelu", "gelu_tanh"]), "gated": rng.random() < 0.25,
         "residual": rng.choice([None, y, "f32"]), "y": y}
    while c["K"] * c["N"] > 8192 * 28672:  # no more weights than the largest listed case
        c["N"] //= 2
    while c["M"] * c["K"] * c["N"] > 2048 * 8192 * 28672:
        c["M"] //= 2
    c["N"] += c["N"] % 2 if c["gated"] else 0
    return c


# -------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _choice_bytes(g, counts, width, shape):
    """Random bytes of codes of ``width`` bits; code c is drawn counts[c] times in sum(counts)."""
    codes = torch.tensor([c for c, n in enumerate(counts) for _ in range(n)])
    n, per = len(codes), 8 // width
    at = torch.arange(n**per)
    table = sum(codes[(at // n**j) % n] << (width * j) for j in range(per)).to(torch.uint8).cuda()
    return table[torch.randint(0, n**per, shape, generator=g, device="cuda")]


def _prepare_weights(c, g):
    N, K, fmt = c["N"], c["K"], c["fmt"]
    s = {"n_out": int(ANCHORS[fmt] * K) if c["anchors"] else 0}
    sigma = 0.02
    if fmt == "2bit":  # the four levels of a normal weight are met about 1 : 2 : 2 : 1
        s["codes"] = _choice_bytes(g, [1, 2, 2, 1], 2, (N, K // 4))
        S = sigma * (1 + 0.15 * _normal(g, N, K // 32))
        s["scales"] = torch.stack([S, 0.1 * sigma * _normal(g, N, K // 32)], -1).half()
    elif fmt == "nf4":  # the levels are quantiles: met about equally often
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = sigma * (2.4 + 0.3 * _normal(g, N, K // 64)).abs()
    else:  # a normal weight on the grid of seventh parts of its group's largest
        s["codes"] = _choice_bytes(g, [0, 1, 1, 1, 2, 3, 4, 4, 4, 4, 4, 3, 2, 1, 1, 1], 4, (N, K // 2))
        s["scales"] = (sigma * (2.1 + 0.3 * _normal(g, N, K // 32)).abs() / 7).half()
    if s["n_out"]:
        n, pad = s["n_out"], -(-s["n_out"] // 8) * 8
        s["out_w"] = torch.zeros(N, pad, dtype=torch.float16, device="cuda")
        s["out_w"][:, :n] = 2 * sigma * _normal(g, N, n)
        if fmt == "2bit":
            idx = torch.rand(K, generator=g, device="cuda").topk(n).indices.sort().values
            s["out_idx"] = idx.to(torch.int32)
            bit = torch.zeros(K, dtype=torch.int64, device="cuda").scatter_(0, idx, 1).view(K // 32, 32)
            word = (bit << torch.arange(32, device="cuda")).sum(-1)
            s["out_mask"] = torch.where(word >= 2**31, word - 2**32, word).to(torch.int32)
        else:  # the first channels of the permuted order; their codes are the zero level
            s["codes"][:, : n // 2] = 0x88
            if n % 2:
                s["codes"][:, n // 2] = s["codes"][:, n // 2] & 0xF0 | 0x08
    return s


def _stand_out(g, x):
    """Some channels of activations are much larger than the others."""
    K = x.shape[1]
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 50)]] *= 8
    return x


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        s["x"] = _normal(g, M, K).to(DT[c["x"]])
        s["residual"] = _stand_out(g, 4 * _normal(g, M, K)).to(DT[c["residual"]]) if c["residual"] else None
        s["weight"] = (1 + 0.2 * _normal(g, K)).to(DT[c["x"]])
        s["perm"] = torch.randperm(K, generator=g, device="cuda").to(torch.int32) if c["perm"] else None
        return s
    if c["op"] == "route":
        x = _normal(g, c["T"], c["E"]) + 0.7 * _normal(g, 1, c["E"])  # some experts are asked for more often
        x = x.to(DT[c["dtype"]])
        x[torch.rand(c["T"], generator=g, device="cuda") < c["pad"]] = -math.inf  # padding goes to no expert
        s["logits"] = x
        s["bias"] = 0.1 * _normal(g, c["E"]) if c["bias"] else None
        return s
    s.update(_prepare_weights(c, g))
    M, K, N = c["M"], c["K"], c["N"]
    width = N // 2 if c["gated"] else N
    x = _stand_out(g, _normal(g, M, K))
    s["x_scales"] = None
    if c["x"] in TOP:  # as a norm leaves them: each row by its largest
        s["x_scales"] = x.abs().amax(1) / TOP[c["x"]]
        x = x / s["x_scales"][:, None]
        x = x.round() if c["x"] == "i8" else x
    s["x"] = x.to(DT[c["x"]])
    s["bias"] = (0.5 * _normal(g, N)).to(DT[c["y"]]) if c["bias"] else None
    s["residual"] = (4 * _normal(g, M, width)).to(DT[c["residual"]]) if c["residual"] else None
    if own:
        from bit_weight_quantized_qw_amd import qw
        fmt = {"2bit": qw.QW_FMT_2BIT_G32, "nf4": qw.QW_FMT_NF4_B64, "int4": qw.QW_FMT_INT4_G32}[c["fmt"]]
        w = s["weights"] = qw.PackedWeight(fmt, N, K, s["n_out"])
        for name in ("codes", "scales", "out_idx", "out_w", "out_mask"):  # the same buffers: nothing is copied
            if s.get(name) is not None:
                t = s[name].view(-1)
                setattr(w, name, t.view(torch.uint8) if name == "scales" else t)
    return s


# ---------------------------------------------------------------- plain form

def _plain_e4m3(v):
    """v (64 bits, within the range) on the grid of e4m3, ties to even: 3 bits behind the first, steps from 2^-9 on."""
    step = torch.exp2((torch.frexp(v).exponent - 1).clamp_min(-6).double() - 3)
    return torch.round(v / step) * step


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["residual"] = h.to(DT[c["residual"]])
    if c["y"] in TOP:
        h = h.double()  # values next to a border of the 8-bit grid
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["weight"].to(h.dtype)
    if s["perm"] is not None:
        y = y[:, s["perm"].long()]
    if c["y"] in TOP:
        scale = (y.abs().amax(-1) / TOP[c["y"]]).float()
        y = y / scale.double()[:, None]
        out["scales"] = scale
        if c["y"] == "i8":
            y = torch.round(y) * scale.double()[:, None]
            return dict(out, y=y.to(DT[c["x"]]))
        y = _plain_e4m3(y).float()
    return dict(out, y=y.to(DT[c["y"]]))


def _plain_weights(s):
    """The weights (N, K) in 32 bits, anchors in place."""
    fmt = s["case"]["fmt"]
    width = 2 if fmt == "2bit" else 4
    shift = torch.arange(0, 8, width, device="cuda", dtype=torch.uint8)
    q = ((s["codes"][..., None] >> shift) & (2**width - 1)).flatten(-2)
    if fmt == "int4":
        level = q.float() - 8
    else:
        level = torch.tensor(CODEBOOK if fmt == "2bit" else _nf4_levels(), device="cuda")[q.int()]
    level = level.unflatten(-1, (-1, GROUP[fmt]))
    scales = s["scales"].float()
    if fmt == "2bit":
        w = (scales[..., :1] * level + scales[..., 1:]).flatten(-2)
    else:
        w = (scales[..., None] * level).flatten(-2)
    n = s["n_out"]
    if n and fmt == "int4":
        w[:, :n] = s["out_w"][:, :n].float()
    elif n:
        w[:, s["out_idx"].long()] = s["out_w"][:, :n].float()
    return w


def _plain_act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ _plain_weights(s).t()
    if s["x_scales"] is not None:
        z = z * s["x_scales"][:, None]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if c["gated"]:
        gate, up = z.chunk(2, -1)
        y = _plain_act(gate, c["act"]) * up
    else:
        y = _plain_act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DT[c["y"]])


def _plain_route(s):
    c, x = s["case"], s["logits"].double()  # the order of values next to each other
    T, E, k, n = c["T"], c["E"], c["k"], c["groups"]
    here = x > -math.inf
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-1e300))
        score = e / e.sum(-1, keepdim=True).clamp_min(1e-300)
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(here, choice, -math.inf)
    if n > 1:
        by = torch.sort(choice.view(T, n, E // n), dim=-1, descending=True).values
        value = by[..., 0]
        if c["by"] == "top2" and E // n > 1:
            value = torch.where(by[..., 1] > -math.inf, value + by[..., 1], value)
        best = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, : c["top_groups"]]
        kept = torch.zeros(T, n, dtype=torch.bool, device="cuda").scatter_(1, best, True)
        choice = torch.where(kept.repeat_interleave(E // n, 1), choice, -math.inf)
    top = torch.sort(choice, dim=-1, descending=True, stable=True)
    ids, taken = top.indices[:, :k], top.values[:, :k] > -math.inf
    w = torch.where(taken, score.gather(1, ids), 0.0)
    if c["norm"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
    ids = torch.where(taken, ids, -1).to(torch.int32)
    key = torch.where(ids < 0, E, ids.long()).view(-1)
    rows = torch.sort(key, stable=True).indices.to(torch.int32)
    count = (key[:, None] == torch.arange(E, device="cuda")).sum(0)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
    return {"ids": ids, "weights": (w * c["scale"]).float(), "offsets": offsets, "rows": rows}


def run(state):
    s = state
    c = s["case"]
    if own:
        from bit_weight_quantized_qw_amd import qw
        if c["op"] == "norm":
            n = qw.qw_rmsnorm(s["x"], s["weight"], 1e-6, residual=s["residual"], perm=s["perm"], out_dtype=DT[c["y"]])
            out = {"y": n.y}
            if n.residual is not None:
                out["residual"] = n.residual
            if n.scales is not None:
                out["scales"] = n.scales
            if c["y"] == "i8":
                out["y"] = (n.y * n.scales[:, None]).to(DT[c["x"]])
            return out
        if c["op"] == "linear":
            return qw.qgemm_linear(s["weights"], s["x"], bias=s["bias"], act=c["act"], gated=c["gated"], residual=s["residual"],
                                   x_scales=s["x_scales"], out_dtype=DT[c["y"]])
        r = qw.qw_route_scored(s["logits"], c["k"], score=c["score"], bias=s["bias"], n_groups=c["groups"], top_groups=c["top_groups"],
                               group_by=c["by"], normalize=c["norm"], scale=c["scale"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.groups.offsets, "rows": r.groups.rows}
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "linear":
        return _plain_linear(s)
    return _plain_route(s)


# ---------------------------------------------------------------- definition

def _exact_grid(v, kind):
    """The nearest number of an 8-bit type, ties to the one whose last bit is 0."""
    if kind == "i8":
        grid = torch.arange(-127.0, 128.0, dtype=torch.float64, device="cuda")
        even = torch.arange(-127, 128, device="cuda") % 2 == 0
    else:
        code = torch.arange(127, device="cuda")  # 0x00 .. 0x7E: the finite numbers that are not negative
        e, m = code // 8, code % 8
        up = torch.where(e > 0, (8 + m) * 2.0 ** (e - 10).double(), m * 2.0**-9).double()
        grid, even = torch.cat([-up.flip(0)[:-1], up]), torch.cat([(code % 2 == 0).flip(0)[:-1], code % 2 == 0])
    hi = torch.searchsorted(grid, v).clamp(1, len(grid) - 1)
    below, above = v - grid[hi - 1], grid[hi] - v
    return torch.where((above < below) | ((above == below) & even[hi]), grid[hi], grid[hi - 1])


def _exact_norm(c, s):
    h = s["x"].double()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].double()
        out["residual"] = h
    y = h * s["weight"].double() / ((h**2).sum(1) / c["K"] + 1e-6).sqrt()[:, None]
    if s["perm"] is not None:
        y = torch.index_select(y, 1, s["perm"].long())
    if c["y"] in TOP:
        out["scales"] = y.abs().max(1).values / TOP[c["y"]]
        y = _exact_grid(y / out["scales"][:, None], c["y"])
        if c["y"] == "i8":
            y = y * out["scales"][:, None]
    return dict(out, y=y)


def _exact_weight(c, s, rows):
    """Some of the rows of the weights (N, K) in 64 bits, from a table of each byte's values."""
    fmt, K, n = c["fmt"], c["K"], s["n_out"]
    width = 2 if fmt == "2bit" else 4
    if fmt == "int4":
        level = torch.arange(-8.0, 8.0, dtype=torch.float64)
    else:  # the constants are 32-bit numbers
        level = torch.tensor(CODEBOOK if fmt == "2bit" else _nf4_levels(), dtype=torch.float32).double()
    byte = torch.arange(256)
    table = torch.stack([level[(byte // 2 ** (width * j)) % 2**width] for j in range(8 // width)], 1).cuda()
    w = table[s["codes"][rows].int()].reshape(-1, K)
    sc = s["scales"][rows].double().repeat_interleave(GROUP[fmt], 1)
    w = w * sc[..., 0] + sc[..., 1] if fmt == "2bit" else w * sc
    if n:
        at = torch.arange(n, device="cuda") if fmt == "int4" else s["out_idx"].long()
        w[:, at] = s["out_w"][rows][:, :n].double()
    return w


def _exact_linear(c, s):
    N, x = c["N"], s["x"].double()
    if s["x_scales"] is not None:
        x = x * s["x_scales"].double()[:, None]
    z = torch.cat([x @ _exact_weight(c, s, slice(n, n + 4096)).t() for n in range(0, N, 4096)], 1)
    if s["bias"] is not None:
        z += s["bias"].double()
    g = z[:, : N // 2] if c["gated"] else z
    if c["act"] == "relu":
        a = torch.where(g > 0, g, 0.0)
    elif c["act"] == "silu":
        a = g * torch.sigmoid(g)
    elif c["act"] == "gelu":
        a = 0.5 * g * torch.special.erfc(-g / 2**0.5)
    elif c["act"] == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
        a = g * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (g + 0.044715 * g**3))
    else:
        a = g
    if c["gated"]:
        a = a * z[:, N // 2:]
    return a if s["residual"] is None else a + s["residual"].double()


def _exact_route(c, s):
    x = s["logits"].double()
    T, E, n = c["T"], c["E"], c["groups"]
    taken = torch.arange(T, device="cuda")
    if c["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(x, 1)
    p = torch.where(x > -math.inf, p, 0.0)
    left = p + (0.0 if s["bias"] is None else s["bias"].double())
    left = torch.where(x > -math.inf, left, -math.inf)

    def take(v):  # the first of the largest of each row, -1 where there is none; taken out of v
        best = v.amax(1, keepdim=True)
        first = torch.where((v == best) & (best > -math.inf), torch.arange(v.shape[1], device="cuda"), v.shape[1]).amin(1)
        v[taken, first.clamp_max(v.shape[1] - 1)] = -math.inf
        return torch.where(first < v.shape[1], first, -1), best[:, 0]

    if n > 1:
        value = torch.zeros(T, n, dtype=torch.float64, device="cuda")
        for g in range(n):
            run_of = left[:, g * (E // n): (g + 1) * (E // n)].clone()
            value[:, g] = take(run_of)[1]
            if c["by"] == "top2":
                second = take(run_of)[1]
                value[:, g] += torch.where(second > -math.inf, second, 0.0)
        kept = torch.zeros(T, n + 1, dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):
            kept[taken, take(value)[0]] = True  # -1: the last column, of no group
        left = torch.where(kept[:, :n].repeat_interleave(E // n, 1), left, -math.inf)
    ids = torch.stack([take(left)[0] for _ in range(c["k"])], 1)
    w = torch.where(ids >= 0, p.gather(1, ids.clamp_min(0)), 0.0)
    if c["norm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": None, "weights": w * c["scale"], "offsets": None, "rows": None}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "route": _exact_route}[c["op"]](c, s)


# ---------------------------------------------------------------------- work

SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "i8": 1, None: 0}


def work(case):
    c = case
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        a_row = K * (SIZE[c["x"]] + 2 * SIZE[c["residual"]] + SIZE[c["y"]]) + (4 if c["y"] in TOP else 0)
        return {"bytes": M * a_row + K * (SIZE[c["x"]] + (4 if c["perm"] else 0)), "flops": 6 * M * K}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * (E * SIZE[c["dtype"]] + k * 12) + 4 * (E + 1) + (4 * E if c["bias"] else 0), "flops": T * E * 6}
    M, K, N = c["M"], c["K"], c["N"]
    bits = {"2bit": 2 + 1, "nf4": 4 + 0.5, "int4": 4 + 0.5}[c["fmt"]]
    n_out = int(ANCHORS[c["fmt"]] * K) if c["anchors"] else 0
    width = N // 2 if c["gated"] else N
    rows = M * (K * SIZE[c["x"]] + width * (SIZE[c["y"]] + SIZE[c["residual"]]))
    return {"bytes": N * (K * bits / 8 + 2 * n_out) + rows + (N * SIZE[c["y"]] if c["bias"] else 0), "flops": 2 * M * K * N}
