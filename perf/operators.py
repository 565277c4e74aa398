"""Cases of two operators beside the MoE + multi-LoRA layer, their plain forms and their exact values.

route   routing by softmax or sigmoid scores, with a per-expert selection bias for load balance,
        expert groups, top-k, renormalised and scaled weights, and the (expert, adapter) sort
dense   one dense projection with segmented multi-LoRA, bias, activation (or SiLU-and-mul) and
        residual: y = act(x W^T + bias + c (x A) B) + residual

own False: elementary torch operations in 32 bits (64 for the scores that decide a selection);
own True: the calls that a user makes of moe_lora_b200.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------- cases

def _route(name, M, E, k, H, L, score, biased, n_group, topk_group, rule, renorm, scale, given, logits=False):
    return {"name": name, "op": "route", "M": M, "E": E, "k": k, "H": H, "L": L, "score": score, "biased": biased,
            "n_group": n_group, "topk_group": topk_group, "rule": rule, "renorm": renorm, "scale": scale,
            "given": given, "logits": logits}


def _dense(name, T, h_in, h_out, L, r, dtype, act, bias, residual, none_frac=0.0):
    return {"name": name, "op": "dense", "T": T, "h_in": h_in, "h_out": h_out, "L": L, "r": r, "dtype": dtype,
            "act": act, "bias": bias, "residual": residual, "none_frac": none_frac}


def listed():
    return [
        # a request's next token through the router of the bf16 decode layer: latency alone
        _route("route one token", 1, 64, 8, 2048, 8, "softmax", False, 1, 1, "max", True, 1.0, False),
        # a decode batch on the e4m3 decode layer's sizes, balanced by a selection bias, four groups of
        # eight; the logits are kept for the load statistics
        _route("route decode", 64, 128, 8, 7168, 32, "sigmoid", True, 8, 4, "top2", True, 2.5, False, True),
        # logits that another program computed (a fused norm and router), an odd batch, 10 groups of 16
        _route("route given odd", 777, 160, 6, 0, 5, "softmax", True, 10, 3, "max", False, 1.0, True),
        # the prefill layer's router with one sigmoid score per expert
        _route("route prefill", 4096, 128, 8, 4096, 16, "sigmoid", True, 1, 1, "max", True, 1.0, False),
        # the largest prompt batch on the largest router: 256 experts in 8 groups, logits kept
        _route("route large", 16384, 256, 8, 7168, 16, "sigmoid", True, 8, 4, "top2", True, 2.5, False, True),
        # the fp32 projection of 64 tokens with its adapters, a GELU and the block's residual
        _dense("dense f32", 64, 512, 512, 4, 16, "f32", "gelu", True, True),
        # one token of one tenant through the dense projection 4096 -> 11008
        _dense("dense one token", 1, 4096, 11008, 32, 16, "bf16", "silu", True, False),
        # a decode batch of 64 tokens of up to 32 tenants through a gated gate_up
        _dense("dense decode gate_up", 64, 4096, 11008, 32, 16, "bf16", "silu_and_mul", False, False),
        # ... and its down projection, added to the residual stream
        _dense("dense decode down", 64, 11008, 4096, 32, 16, "bf16", "none", False, True),
        # a small mixed batch at odd sizes, part of it without an adapter
        _dense("dense odd", 203, 2056, 1000, 5, 8, "bf16", "gelu", True, False, 0.3),
        # prompts of 16 tenants through a projection with bias and tanh GELU
        _dense("dense prefill", 4096, 4096, 11008, 16, 64, "bf16", "gelu_tanh", True, False),
        # the largest: prompts of 16 tenants, some tokens without one, through a gated gate_up
        _dense("dense large", 8192, 4096, 11008, 16, 64, "bf16", "silu_and_mul", False, False, 0.1),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    if rng.random() < 0.45:
        E = rng.choice([8, 20, 64, 96, 128, 160, 200, 256])
        groups = rng.random() < 0.5
        n_group = rng.choice([4, 8] if E % 8 == 0 else [2, 4]) if groups else 1
        topk_group = rng.randint(max(1, n_group // 2), n_group)
        k = rng.randint(1, min(10, topk_group * (E // n_group)))
        given = rng.random() < 0.25
        score = rng.choice(["softmax", "sigmoid"])
        return _without_name(_route(
            "", _log(rng, 1, 16384), E, k, 0 if given else _log(rng, 256, 7168, 8), rng.choice([0, 1, 5, 8, 32, 64]),
            score, rng.random() < 0.6, n_group, topk_group, rng.choice(["max", "top2"]), rng.random() < 0.7,
            rng.choice([1.0, 2.5]), given, rng.random() < 0.3))
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "silu_and_mul"])
    bias, residual = rng.random() < 0.5, rng.random() < 0.5
    none_frac = rng.choice([0.0, 0.0, 0.3])
    if rng.random() < 0.2:
        return _without_name(_dense("", _log(rng, 1, 512), _log(rng, 128, 2048, 8), _log(rng, 128, 2048, 8),
                                    rng.choice([0, 4, 9]), rng.choice([8, 16, 64]), "f32", act, bias, residual,
                                    none_frac))
    h_in, h_out = _log(rng, 512, 11008, 8), _log(rng, 512, 11008, 8)
    most = 8192 * 4096 * 22016 // (h_in * h_out * (2 if act == "silu_and_mul" else 1))
    T = _log(rng, 1, min(8192, most * 9 // 10))
    return _without_name(_dense("", T, h_in, h_out, rng.choice([0, 1, 7, 16, 32]), rng.choice([8, 16, 32, 64, 128]),
                                "bf16", act, bias, residual, none_frac))


def _without_name(case):
    return {k: v for k, v in case.items() if k != "name"}


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _grid(g, shape, std, bits):
    """Normal values of the given deviation on a grid of 2^-bits, within 4 deviations."""
    v = torch.randn(shape, generator=g, device=DEV).clamp_(-4, 4) * std
    return torch.round(v * 2.0 ** bits) * 2.0 ** -bits


def _adapter_ids(g, n, L, none_frac):
    """Adapter of each token: the i-th with a probability that falls as (i + 1)^-1.1; -1 = none."""
    if L == 0:
        return torch.full((n,), -1, dtype=torch.int32, device=DEV)
    p = (torch.arange(L, device=DEV, dtype=torch.float64) + 1) ** -1.1
    ids = torch.multinomial(p, n, replacement=True, generator=g).to(torch.int32)
    return torch.where(torch.rand(n, generator=g, device=DEV) < none_frac, -torch.ones_like(ids), ids)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "route":
        M, E, H, L = case["M"], case["E"], case["H"], case["L"]
        s = {"case": case, "adapter_ids": _adapter_ids(g, M, L, 0.1), "x": None, "w_router": None, "logits": None,
             "score_bias": None}
        if case["given"]:
            s["logits"] = torch.randn((M, E), generator=g, device=DEV)
        else:
            # normalised activations and a router weight on grids (1/16, and about 1/24 of the
            # weight's deviation): every partial sum of a logit is then exact in 32 bits in any
            # order, so the chosen experts can be compared one by one
            s["x"] = _grid(g, (M, H), 1.0, 4).to(torch.bfloat16)
            bits = math.ceil(math.log2(24 * math.sqrt(H)))
            s["w_router"] = _grid(g, (E, H), H ** -0.5, bits).to(torch.bfloat16)
        if case["biased"]:  # what a balancing rule has added up: small steps either way
            s["score_bias"] = torch.randn((E,), generator=g, device=DEV) * 0.05
        return s
    T, K, N, L, r = case["T"], case["h_in"], case["h_out"], case["L"], case["r"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    rows = 2 * N if case["act"] == "silu_and_mul" else N

    def normal(shape, std):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)

    s = {"case": case, "x": normal((T, K), 1.0), "w": normal((rows, K), K ** -0.5), "a": None, "b": None,
         "seg_offsets": None, "seg_adapter": None,
         "bias": normal((rows,), 0.5) if case["bias"] else None,
         "residual": normal((T, N), 1.0) if case["residual"] else None}
    if L > 0:
        ids = torch.sort(_adapter_ids(g, T, L, case["none_frac"])).values
        ad, n = torch.unique_consecutive(ids, return_counts=True)  # tokens of one adapter side by side
        s["seg_adapter"] = ad.to(torch.int32)
        s["seg_offsets"] = torch.cat([torch.zeros(1, device=DEV, dtype=torch.int64), n.cumsum(0)]).to(torch.int32)
        s["a"], s["b"] = normal((L, r, K), K ** -0.5), normal((L, r, rows), r ** -0.5)
    return s


LORA_SCALE = 0.5


# ------------------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    if own:
        import moe_lora_b200 as ml
        if c["op"] == "route":
            o = ml.route_scored(s["adapter_ids"], c["k"], c["L"], x=s["x"], w_router=s["w_router"],
                                logits_in=s["logits"], score=c["score"], score_bias=s["score_bias"],
                                n_group=c["n_group"], topk_group=c["topk_group"], group_rule=c["rule"],
                                renormalize=c["renorm"], scale=c["scale"], want_logits=c["logits"])
            got = (o["topk_ids"], o["topk_w"], o["sorted_pairs"], o["seg_offsets"])
            return got + (o["logits"],) if c["logits"] else got
        return ml.dense_lora_fused(s["x"], s["w"], s["a"], s["b"], s["seg_offsets"], s["seg_adapter"],
                                   bias=s["bias"], activation=c["act"], residual=s["residual"],
                                   lora_scale=LORA_SCALE)
    return _route_plain(s, c) if c["op"] == "route" else _dense_plain(s, c)


def _route_plain(s, c):
    E, k, L, G = c["E"], c["k"], c["L"], c["n_group"]
    logits = s["logits"] if c["given"] else s["x"].float() @ s["w_router"].float().t()
    M = logits.shape[0]
    l = logits.double()  # the scores decide which experts are chosen: 64 bits at the borders
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.max(1, keepdim=True).values)
        score = e / e.sum(1, keepdim=True)
    sel = score if s["score_bias"] is None else score + s["score_bias"].double()
    if G > 1:
        of = torch.sort(sel.view(M, G, E // G), dim=2, descending=True).values
        group = of[:, :, 0] if c["rule"] == "max" or E == G else of[:, :, 0] + of[:, :, 1]
        best = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : c["topk_group"]]
        keep = torch.zeros((M, G), dtype=torch.bool, device=l.device).scatter(1, best, True)
        sel = torch.where(keep[:, :, None].expand(M, G, E // G).reshape(M, E), sel, -math.inf)
    ids = torch.sort(sel, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    a = s["adapter_ids"].long()
    key = (ids * (L + 1) + torch.where(a >= 0, a, L)[:, None]).reshape(-1)
    pairs = torch.sort(key, stable=True).indices
    count = torch.zeros(E * (L + 1) + 1, dtype=torch.int64, device=l.device)
    count.index_add_(0, key + 1, torch.ones_like(key))
    got = (ids.int(), (w * c["scale"]).float(), pairs.int(), count.cumsum(0).int())
    return got + (logits.clone() if c["given"] else logits,) if c["logits"] else got


def _dense_plain(s, c):
    x = s["x"].float()
    h = x @ s["w"].float().t()
    if s["bias"] is not None:
        h = h + s["bias"].float()
    if c["L"] > 0:
        T, L, r = c["T"], c["L"], c["r"]
        n = s["seg_offsets"][1:] - s["seg_offsets"][:-1]
        ad = torch.repeat_interleave(s["seg_adapter"], n, output_size=T)
        z = (x @ s["a"].float().reshape(L * r, -1).t()).view(T, L, r)
        z = torch.where((ad[:, None] == torch.arange(L, device=x.device))[:, :, None], z, 0.0) * LORA_SCALE
        h = h + z.reshape(T, L * r) @ s["b"].float().reshape(L * r, -1)
    act = c["act"]
    if act == "relu":
        h = torch.where(h > 0, h, 0.0)
    elif act == "gelu":
        h = 0.5 * h * (1 + torch.erf(h * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        h = 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))
    elif act == "silu":
        h = h / (1 + torch.exp(-h))
    elif act == "silu_and_mul":
        g, u = h[:, : c["h_out"]], h[:, c["h_out"]:]
        h = g / (1 + torch.exp(-g)) * u
    if s["residual"] is not None:
        h = h + s["residual"].float()
    return h.to(s["x"].dtype)


# ------------------------------------------------------------------------------- what a pass cannot do without

def work(c):
    if c["op"] == "route":
        M, E, H = c["M"], c["E"], c["H"]
        read = 4 * M * E if c["given"] else 2 * H * (M + E)
        out = 8 * M * c["k"] + 4 * M * c["k"] + 4 * (E * (c["L"] + 1) + 1) + (4 * M * E if c["logits"] else 0)
        return {"bytes": read + 4 * M + out, "flops": 0 if c["given"] else 2 * M * E * H}
    T, K, N, L, r = c["T"], c["h_in"], c["h_out"], c["L"], c["r"]
    size = 4 if c["dtype"] == "f32" else 2
    rows = 2 * N if c["act"] == "silu_and_mul" else N
    used = min(L, T)  # at most one adapter per token
    n = T * K + rows * K + T * N + used * r * (K + rows) + (rows if c["bias"] else 0) + (T * N if c["residual"] else 0)
    return {"bytes": size * n, "flops": 2 * T * K * rows + (2 * T * r * (K + rows) if L else 0)}


# ------------------------------------------------------------------------------- exact values

def exact(case, seed):
    s = prepare(case, seed)
    return _route_exact(s, case) if case["op"] == "route" else _dense_exact(s, case)


def _route_exact(s, c):
    E, k, L, G, M = c["E"], c["k"], c["L"], c["n_group"], c["M"]
    if c["given"]:
        l = s["logits"].double().cpu().numpy()
    else:
        l = torch.einsum("mh,eh->me", s["x"].double(), s["w_router"].double()).cpu().numpy()
    if c["score"] == "sigmoid":
        p = 0.5 * (1 + np.tanh(0.5 * l))
    else:
        p = np.exp(l - np.logaddexp.reduce(l, axis=1)[:, None])
    want = p + (0 if s["score_bias"] is None else s["score_bias"].double().cpu().numpy())
    if G > 1:
        by = np.sort(want.reshape(M, G, -1), axis=2)
        top = by[:, :, -1] + (by[:, :, -2] if c["rule"] == "top2" and E > G else 0)
        rank = np.argsort(np.argsort(-top, axis=1, kind="stable"), axis=1, kind="stable")
        want = np.where(np.repeat(rank < c["topk_group"], E // G, axis=1), want, -np.inf)
    ids = np.argsort(-want, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    a = s["adapter_ids"].cpu().numpy().astype(np.int64)
    key = (ids * (L + 1) + np.where(a < 0, L, a)[:, None]).ravel()
    off = np.searchsorted(np.sort(key), np.arange(E * (L + 1) + 1), side="left")
    got = (ids.astype(np.int32), w * c["scale"], np.argsort(key, kind="stable").astype(np.int32),
           off.astype(np.int32))
    return got + (l,) if c["logits"] else got


def _dense_exact(s, c):
    x, w = s["x"].double(), s["w"].double()
    h = torch.einsum("tk,nk->tn", x, w)
    if c["L"] > 0:
        off, ad = s["seg_offsets"].tolist(), s["seg_adapter"].tolist()
        for i, a in enumerate(ad):
            if a >= 0:
                rows = slice(off[i], off[i + 1])
                h[rows] += LORA_SCALE * (x[rows] @ s["a"][a].double().t() @ s["b"][a].double())
    if s["bias"] is not None:
        h += s["bias"].double()
    f = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.sigmoid(v),
         "gelu": lambda v: v * 0.5 * torch.erfc(-v / math.sqrt(2)),
         "gelu_tanh": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)),
         "silu_and_mul": lambda v: v[:, : c["h_out"]] * torch.sigmoid(v[:, : c["h_out"]]) * v[:, c["h_out"]:]}
    h = f[c["act"]](h)
    if s["residual"] is not None:
        h = h + s["residual"].double()
    return h
