"""The operators whose rows of one batch take different matrices, as cases to measure.

Four operators: ``route`` (a router's top-k and the grouping of the rows by
expert), ``experts`` (the product of every group with its expert's packed
weight, plain or gated), ``combine`` (the same product with the weighted sum
of a token's experts) and ``lora`` (the low-rank adapters of many requests
added to a shared projection's output).

``run`` computes a case in its plain form (elementary torch operations in 32
bits) or, where ``own`` is true, by the library's calls. ``exact`` computes
the definition in 64 bits.
"""

import math
from statistics import NormalDist

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODEBOOK = [-1.52, -0.45, 0.45, 1.52]
GROUP = {"2bit": 32, "nf4": 64, "int4": 32}       # weights per scale
ANCHORS = {"2bit": 0.035, "nf4": 0.0, "int4": 0.01}  # share of the channels kept in fp16


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
        # a decode step of a batch of 48 requests, a tenth of the slots padding
        {"name": "route_decode", "op": "route", "T": 48, "E": 64, "k": 8, "dtype": "f32", "norm": True, "pad": 0.1},
        # a prefill of 16384 tokens over many experts
        {"name": "route_prefill", "op": "route", "T": 16384, "E": 128, "k": 8, "dtype": "bf16", "norm": False, "pad": 0.0},
        # one token's gate and up projections in eight of 64 small experts: latency
        {"name": "experts_token", "op": "experts", "T": 1, "E": 64, "k": 8, "K": 2048, "N": 2816, "fmt": "2bit",
         "anchors": False, "dtype": "f16", "swiglu": True, "pad": 0.0},
        # a decode batch over a few large experts: every weight streams once
        {"name": "experts_decode", "op": "experts", "T": 40, "E": 16, "k": 2, "K": 4096, "N": 8192, "fmt": "nf4",
         "anchors": False, "dtype": "f16", "swiglu": False, "pad": 0.05},
        # a short ragged prefill: some 40 rows an expert, an odd number of columns, fp16 anchors
        {"name": "experts_ragged", "op": "experts", "T": 333, "E": 32, "k": 4, "K": 2048, "N": 1501, "fmt": "int4",
         "anchors": True, "dtype": "bf16", "swiglu": False, "pad": 0.03},
        # a prefill's gate and up projections in 64 small experts
        {"name": "experts_gated", "op": "experts", "T": 2000, "E": 64, "k": 6, "K": 2048, "N": 2816, "fmt": "int4",
         "anchors": False, "dtype": "bf16", "swiglu": True, "pad": 0.0},
        # a long prefill in eight large experts: the matrix cores' rate
        {"name": "experts_prefill", "op": "experts", "T": 4096, "E": 8, "k": 2, "K": 4096, "N": 14336, "fmt": "2bit",
         "anchors": False, "dtype": "bf16", "swiglu": False, "pad": 0.0},
        # the down projections of a small decode batch, with anchors, summed per token
        {"name": "combine_decode", "op": "combine", "T": 17, "E": 64, "k": 8, "K": 1408, "N": 2048, "fmt": "2bit",
         "anchors": True, "dtype": "f16", "pad": 0.1},
        # the down projections of a prefill
        {"name": "combine_prefill", "op": "combine", "T": 2048, "E": 16, "k": 4, "K": 2816, "N": 5120, "fmt": "nf4",
         "anchors": False, "dtype": "bf16", "pad": 0.02},
        # one request's adapter beside one projection: latency
        {"name": "lora_token", "op": "lora", "M": 1, "n": 32, "K": 4096, "N": 4096, "r": 16, "dtype": "f16",
         "base": "f32", "run_len": 1, "none": 0.0},
        # a decode batch of 64 requests over 32 adapters, some requests without one
        {"name": "lora_decode", "op": "lora", "M": 64, "n": 32, "K": 5120, "N": 13824, "r": 32, "dtype": "f16",
         "base": "f32", "run_len": 1, "none": 0.1},
        # the prompts of some requests, a run of rows each
        {"name": "lora_prefill", "op": "lora", "M": 4001, "n": 8, "K": 4096, "N": 11008, "r": 64, "dtype": "bf16",
         "base": "bf16", "run_len": 300, "none": 0.1},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "combine", "lora"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256])
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, 8), "dtype": rng.choice(["f32", "bf16", "f16"]),
                "norm": rng.random() < 0.5, "pad": rng.choice([0.0, 0.1])}
    if op == "lora":
        n, dtype = _log(rng, 1, 64), rng.choice(["f16", "bf16"])
        M = _log(rng, 1, 4096)
        return {"op": op, "M": M, "n": n, "K": _log(rng, 512, 8192, 64), "N": _log(rng, 500, 16000), "r": rng.choice([8, 16, 24, 32, 64, 128]),
                "dtype": dtype, "base": rng.choice([dtype, "f32"]), "run_len": 1 if M <= 128 else rng.randint(1, 600),
                "none": rng.choice([0.0, 0.2])}
    E = rng.choice([4, 8, 16, 40, 64])
    K, N = _log(rng, 512, 4096, 64), _log(rng, 500, 8192)
    while E * K * N > 8 * 4096 * 14336:  # no more weights than the largest listed case
        E //= 2
    fmt = rng.choice(["2bit", "nf4", "int4"])
    c = {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(E, 8)), "K": K, "N": N, "fmt": fmt,
         "anchors": fmt != "nf4" and rng.random() < 0.5, "dtype": rng.choice(["f16", "bf16"])}
    while c["T"] * c["k"] * K * N > 8192 * 4096 * 14336:
        c["T"] //= 2
    if op == "experts":
        c["swiglu"] = rng.random() < 0.3
        c["N"] += c["N"] % 2 if c["swiglu"] else 0
    return dict(c, pad=rng.choice([0.0, 0.1]))


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


def _group(ids, count):
    """Rows in the order of their ids, those of one id ascending, rows without one (-1) behind all
    others, and the place where each id's rows begin: what a grouping call leaves."""
    key = torch.where(ids < 0, count, ids.long())
    rows = torch.sort(key, stable=True).indices.to(torch.int32)
    n = (key[:, None] == torch.arange(count, device=key.device)).sum(0)
    return torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32), rows


def _prepare_weights(c, g):
    E, N, K, fmt = c["E"], c["N"], c["K"], c["fmt"]
    s = {"n_out": int(ANCHORS[fmt] * K) if c["anchors"] else 0}
    sigma = 0.02
    if fmt == "2bit":  # the four levels of a normal weight are met about 1 : 2 : 2 : 1
        s["codes"] = _choice_bytes(g, [1, 2, 2, 1], 2, (E, N, K // 4))
        S = sigma * (1 + 0.15 * _normal(g, E, N, K // 32))
        s["scales"] = torch.stack([S, 0.1 * sigma * _normal(g, E, N, K // 32)], -1).half()
    elif fmt == "nf4":  # the levels are quantiles: met about equally often
        s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = sigma * (2.4 + 0.3 * _normal(g, E, N, K // 64)).abs()
    else:  # a normal weight on the grid of seventh parts of its group's largest
        s["codes"] = _choice_bytes(g, [0, 1, 1, 1, 2, 3, 4, 4, 4, 4, 4, 3, 2, 1, 1, 1], 4, (E, N, K // 2))
        s["scales"] = (sigma * (2.1 + 0.3 * _normal(g, E, N, K // 32)).abs() / 7).half()
    if s["n_out"]:
        n, pad = s["n_out"], -(-s["n_out"] // 8) * 8
        s["out_w"] = torch.zeros(E, N, pad, dtype=torch.float16, device="cuda")
        s["out_w"][..., :n] = 2 * sigma * _normal(g, E, N, n)
        if fmt == "2bit":
            idx = torch.rand(E, K, generator=g, device="cuda").topk(n, 1).indices.sort(1).values
            s["out_idx"] = idx.to(torch.int32)
            bit = torch.zeros(E, K, dtype=torch.int64, device="cuda").scatter_(1, idx, 1).view(E, K // 32, 32)
            word = (bit << torch.arange(32, device="cuda")).sum(-1)
            s["out_mask"] = torch.where(word >= 2**31, word - 2**32, word).to(torch.int32)
        else:  # the first channels of the permuted order; their codes are the zero level
            s["codes"][..., : n // 2] = 0x88
            if n % 2:
                s["codes"][..., n // 2] = s["codes"][..., n // 2] & 0xF0 | 0x08
    return s


def _logits(c, g):
    x = _normal(g, c["T"], c["E"]) + 0.7 * _normal(g, 1, c["E"])  # some experts are asked for more often
    x = x.to(DT[c["dtype"]])
    x[torch.rand(c["T"], generator=g, device="cuda") < c["pad"]] = -math.inf  # padding goes to no expert
    return x


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = DT[c["dtype"]]
    if c["op"] == "route":
        return {"case": c, "logits": _logits(c, g)}
    if c["op"] == "lora":
        M, n, K, N, r = c["M"], c["n"], c["K"], c["N"], c["r"]
        s = {"case": c, "x": _normal(g, M, K).to(dt), "base": _normal(g, M, N).to(DT[c["base"]]),
             "A": (_normal(g, n, r, K) / math.sqrt(K)).to(dt), "B": (_normal(g, n, N, r) / math.sqrt(r)).to(dt),
             "scale": 0.5 + torch.rand(n, generator=g, device="cuda")}
        runs = -(-M // c["run_len"])
        ids = torch.randint(0, n, (runs,), generator=g, device="cuda")
        ids[torch.rand(runs, generator=g, device="cuda") < c["none"]] = -1
        s["ids"] = ids.repeat_interleave(c["run_len"])[:M].to(torch.int32)
        s["offsets"], s["rows"] = _group(s["ids"], n)  # once for a step, for all its layers
        if own:
            from bit_weight_quantized_qw_amd import qw
            s["adapters"] = qw.Adapters(s["A"], s["B"], s["scale"])  # the same buffers: nothing is copied
            s["groups"] = qw.RowGroups(s["offsets"], s["rows"])
        return s
    s = {"case": c, **_prepare_weights(c, g)}
    T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
    p, ids = torch.softmax(_logits(c, g).float(), -1).topk(k, -1)
    s["ids"] = torch.where(p > 0, ids, -1).to(torch.int32)
    s["weights"] = torch.where(p > 0, p / p.sum(-1, keepdim=True), 0.0)
    s["offsets"], s["rows"] = _group(s["ids"].view(-1), E)
    count = s["offsets"].diff()
    s["filled"], s["cap"] = int(count.sum()), max(1, int(count.max()))  # for the plain form's padded batch
    if c["op"] == "experts":
        x = _normal(g, T, K)
        out = N // 2 if c["swiglu"] else N
        s["out"] = torch.zeros(T * k, out, dtype=dt, device="cuda")  # rows of no expert stay as they are
    else:
        x = 0.3 * _normal(g, T * k, K)  # the gated activations, in the experts' order
    x[:, torch.randperm(K, generator=g, device="cuda")[: K // 50]] *= 8  # channels that stand out
    s["x"] = x.to(dt)
    if own:
        from bit_weight_quantized_qw_amd import qw
        fmt = {"2bit": qw.QW_FMT_2BIT_G32, "nf4": qw.QW_FMT_NF4_B64, "int4": qw.QW_FMT_INT4_G32}[c["fmt"]]
        s["experts"] = qw.ExpertWeights(fmt, E, N, K, s["n_out"], s["codes"], s["scales"], s.get("out_idx"), s.get("out_w"),
                                        s.get("out_mask"))  # the same buffers: nothing is copied
        s["groups"] = qw.RowGroups(s["offsets"], s["rows"])
    return s


# ---------------------------------------------------------------- plain form

def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    E, k = c["E"], c["k"]
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-3e38))
    top = torch.sort(x, dim=-1, descending=True, stable=True)
    ids, value = top.indices[:, :k], top.values[:, :k]
    taken = value > -math.inf
    w = torch.where(taken, torch.gather(p, 1, ids), 0.0)
    total = (w if c["norm"] else p).sum(-1, keepdim=True)
    ids = torch.where(taken, ids, -1).to(torch.int32)
    offsets, rows = _group(ids.view(-1), E)
    return {"ids": ids, "weights": torch.where(taken, w / total, 0.0), "offsets": offsets, "rows": rows}


def _plain_dequant(s, codes, scales):
    """The weights (e, N, K) of some experts in 32 bits, their anchor channels apart."""
    fmt = s["case"]["fmt"]
    width = 2 if fmt == "2bit" else 4
    shift = torch.arange(0, 8, width, device=codes.device, dtype=torch.uint8)
    q = ((codes[..., None] >> shift) & (2**width - 1)).flatten(-2).long()
    if fmt == "int4":
        level = q.float() - 8
    else:
        level = torch.tensor(CODEBOOK if fmt == "2bit" else _nf4_levels(), device=q.device)[q]
    level = level.unflatten(-1, (-1, GROUP[fmt]))
    scales = scales.float()
    if fmt == "2bit":
        return (scales[..., :1] * level + scales[..., 1:]).flatten(-2)
    return (scales[..., None] * level).flatten(-2)


def _plain_weights(s, e):
    """The weights of the experts e (an index or a slice), anchors in place."""
    w = _plain_dequant(s, s["codes"][e], s["scales"][e])
    n = s["n_out"]
    if not n:
        return w
    out_w = s["out_w"][e][..., :n].float()
    if s["case"]["fmt"] == "int4":
        w[..., :n] = out_w
        return w
    idx = s["out_idx"][e].long()[:, None, :].expand(-1, w.shape[1], -1)
    return w.scatter_(2, idx, out_w)


def _plain_products(s, x):
    """Every filled row's product with its expert's weights, in 32 bits, in the experts' order."""
    E, K = s["case"]["E"], s["case"]["K"]
    at = torch.arange(s["filled"], device=x.device)
    e = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    if s["filled"] < E:  # fewer rows than experts: each row's own weights
        return torch.matmul(_plain_weights(s, e), x[..., None])[..., 0]
    within = at - s["offsets"][e]
    padded = x.new_zeros(E, s["cap"], K)
    padded[e, within] = x
    return torch.matmul(padded, _plain_weights(s, slice(None)).transpose(1, 2))[e, within]


def _plain_experts(s):
    c = s["case"]
    slot = s["rows"][: s["filled"]].long()
    y = _plain_products(s, s["x"][slot // c["k"]].float())
    if c["swiglu"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1 + torch.exp(-gate)) * up
    out = torch.zeros_like(s["out"])
    out[: s["filled"]] = y.to(out.dtype)
    return out


def _plain_combine(s):
    c = s["case"]
    slot = s["rows"][: s["filled"]].long()
    y = torch.zeros(c["T"] * c["k"], c["N"], device="cuda")
    y[slot] = _plain_products(s, s["x"][: s["filled"]].float())
    y = (y.view(c["T"], c["k"], c["N"]) * s["weights"][..., None]).sum(1)
    return y.to(DT[c["dtype"]])


def _plain_lora(s):
    c, ids = s["case"], s["ids"].long()
    n, r, M = c["n"], c["r"], c["M"]
    x, has, a = s["x"].float(), (ids >= 0)[:, None], ids.clamp_min(0)
    if M <= n:  # fewer rows than adapters: each row's own
        t = torch.matmul(s["A"][a].float(), x[..., None])
        d = torch.matmul(s["B"][a].float(), t)[..., 0]
    else:  # all adapters' inner values, of which each row keeps its own
        t = (x @ s["A"].float().view(n * r, -1).t()).view(M, n, r)
        t = t * (torch.arange(n, device=a.device)[None, :, None] == a[:, None, None])
        d = t.view(M, n * r) @ s["B"].float().transpose(1, 2).reshape(n * r, -1)
    y = s["base"].float() + torch.where(has, s["scale"][a][:, None] * d, 0.0)
    return y.to(DT[c["dtype"]])


def run(state):
    s = state
    c = s["case"]
    if own:
        from bit_weight_quantized_qw_amd import qw
        if c["op"] == "route":
            r = qw.qw_route_topk(s["logits"], c["k"], normalize=c["norm"])
            return {"ids": r.ids, "weights": r.weights, "offsets": r.groups.offsets, "rows": r.groups.rows}
        if c["op"] == "experts":
            return qw.qgemm_experts(s["experts"], s["x"], s["groups"], top_k=c["k"], swiglu=c["swiglu"], out=s["out"])
        if c["op"] == "combine":
            return qw.qgemm_experts_combine(s["experts"], s["x"], s["groups"], s["ids"], s["weights"])
        return qw.qw_lora_add(s["adapters"], s["x"], s["groups"], s["base"], out_dtype=DT[c["dtype"]])
    if c["op"] == "route":
        return _plain_route(s)
    if c["op"] == "experts":
        return _plain_experts(s)
    if c["op"] == "combine":
        return _plain_combine(s)
    return _plain_lora(s)


# ---------------------------------------------------------------- definition

def _exact_weight(s, e):
    """Expert e's weights (N, K) in 64 bits, from a table of each byte's values."""
    c = s["case"]
    fmt, N, K, n = c["fmt"], c["N"], c["K"], s["n_out"]
    width = 2 if fmt == "2bit" else 4
    if fmt == "int4":
        level = torch.arange(-8.0, 8.0, dtype=torch.float64)
    else:  # the constants are 32-bit numbers
        level = torch.tensor(CODEBOOK if fmt == "2bit" else _nf4_levels(), dtype=torch.float32).double()
    byte = torch.arange(256)
    table = torch.stack([level[(byte // 2 ** (width * j)) % 2**width] for j in range(8 // width)], 1).cuda()
    w = table[s["codes"][e].long()].reshape(N, K)
    sc = s["scales"][e].double().repeat_interleave(GROUP[fmt], 1)
    w = w * sc[..., 0] + sc[..., 1] if fmt == "2bit" else w * sc
    if n:
        at = torch.arange(n, device=w.device) if fmt == "int4" else s["out_idx"][e].long()
        w[:, at] = s["out_w"][e][:, :n].double()
    return w


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        x = s["logits"].double()
        T, E, k = c["T"], c["E"], c["k"]
        ids = torch.full((T, k), -1, dtype=torch.int64, device="cuda")
        left, rows = x.clone(), torch.arange(T, device="cuda")
        for j in range(k):
            best = left.amax(1, keepdim=True)
            first = torch.where((left == best) & (best > -math.inf), torch.arange(E, device="cuda"), E).amin(1)
            ids[:, j] = torch.where(first < E, first, -1)
            left[rows, first.clamp_max(E - 1)] = -math.inf
        e = torch.where(x > -math.inf, torch.exp(x - x.amax(1, keepdim=True)), 0.0)
        w = torch.where(ids >= 0, e.gather(1, ids.clamp_min(0)), 0.0)
        total = (w if c["norm"] else e).sum(1, keepdim=True)
        return {"ids": None, "weights": torch.where(ids >= 0, w / total, 0.0), "offsets": None, "rows": None}
    if c["op"] == "lora":
        y = s["base"].double()
        for a in range(c["n"]):
            m = (s["ids"] == a).nonzero()[:, 0]
            t = s["x"][m].double() @ s["A"][a].double().t()
            y[m] += s["scale"][a].double() * (t @ s["B"][a].double().t())
        return y
    T, k, N = c["T"], c["k"], c["N"]
    at = [int(v) for v in s["offsets"].cpu()]
    slot = s["rows"].long()
    y = torch.zeros(T * k, N, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        here = slice(at[e], at[e + 1])
        if at[e + 1] > at[e]:
            x = s["x"][slot[here] // k] if c["op"] == "experts" else s["x"][here]
            y[here] = x.double() @ _exact_weight(s, e).t()
    if c["op"] == "experts":
        return torch.sigmoid(y[:, : N // 2]) * y[:, : N // 2] * y[:, N // 2:] if c["swiglu"] else y
    token = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    token.index_add_(0, slot // k, y * s["weights"].view(-1)[slot, None].double())
    return token


# ---------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "route":
        size = {"f32": 4, "bf16": 2, "f16": 2}[c["dtype"]]
        return {"bytes": c["T"] * (c["E"] * size + c["k"] * 12) + 4 * (c["E"] + 1), "flops": c["T"] * c["E"] * 4}
    if c["op"] == "lora":
        M, n, K, N, r = c["M"], c["n"], c["K"], c["N"], c["r"]
        runs = -(-M // c["run_len"]) * (1 - c["none"])
        used = n * (1 - (1 - 1 / n) ** runs)  # adapters that some row takes, in the mean
        base = 4 if c["base"] == "f32" else 2
        return {"bytes": 2 * M * K + 2 * used * r * (K + N) + M * N * (base + 2), "flops": 2 * M * r * (K + N)}
    T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
    T = T * (1 - c["pad"])
    bits = {"2bit": 2 + 1, "nf4": 4 + 0.5, "int4": 4 + 0.5}[c["fmt"]]
    n_out = int(ANCHORS[c["fmt"]] * K) if c["anchors"] else 0
    used = E * (1 - (1 - k / E) ** T)  # experts that some row takes, in the mean
    weights = used * N * (K * bits / 8 + 2 * n_out)
    if c["op"] == "experts":
        return {"bytes": weights + 2 * T * K + 2 * T * k * (N // 2 if c["swiglu"] else N), "flops": 2 * T * k * K * N}
    return {"bytes": weights + 2 * T * k * K + 2 * T * N, "flops": 2 * T * k * K * N}
