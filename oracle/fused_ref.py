"""fp64 reference of scored routing and of the fused dense projection.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Scored routing is the generic form
of the choice of each token's most relevant experts ([vLLM MoE-LoRA page], "Entendendo os
Modelos MoE"); the projection is y = xW + (xA)B ("O Papel da Multi-LoRA") over contiguous
segments ([Punica review page], "提案手法") with everything behind the product in one place.
"""
from __future__ import annotations

import math

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def _finite(v: np.ndarray) -> np.ndarray:
    return np.clip(v, -F32_MAX, F32_MAX)


def scores(logits: np.ndarray, score: str) -> np.ndarray:
    """softmax over the row's numbers, or the logistic function; 0 for a NaN."""
    nan = np.isnan(logits)
    l = _finite(np.where(nan, 0.0, logits))
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            m = np.max(np.where(nan, -F32_MAX, l), axis=1, keepdims=True)
            e = np.where(nan, 0.0, np.exp(np.where(nan, 0.0, l) - m))
            tot = e.sum(1, keepdims=True)
            s = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
    return np.where(nan, 0.0, s)


def route_scored(logits, k, *, score="softmax", score_bias=None, n_group=1, topk_group=1, group_rule="max",
                 renormalize=True, scale=1.0):
    """ids int32 [M, k] and weights fp64 [M, k] of the fp64 definition."""
    M, E = logits.shape
    s = scores(logits, score)
    nan = np.isnan(logits)
    bias = np.zeros(E) if score_bias is None else _finite(np.nan_to_num(np.asarray(score_bias, np.float64), nan=0.0,
                                                                        posinf=F32_MAX, neginf=-F32_MAX))
    by_logit = score_bias is None and not (n_group > 1 and group_rule == "top2")
    if by_logit:
        c = _finite(np.where(nan, 0.0, logits))
    else:
        b = np.zeros(E) if score_bias is None else np.asarray(score_bias, dtype=np.float64)
        nan = nan | np.isnan(b)[None, :]
        c = s + _finite(np.where(np.isnan(b), 0.0, b))[None, :]
    c = np.where(nan, -np.inf, c)
    gs = E // n_group
    ids = np.empty((M, k), dtype=np.int32)
    for t in range(M):
        allowed = list(range(E))
        if n_group > 1:
            top = []
            for g in range(n_group):
                v = sorted(range(g * gs, (g + 1) * gs), key=lambda e: (-c[t, e], e))
                if group_rule == "top2" and gs > 1:
                    # scores and biases summed apart: groups whose two best have the same
                    # scores and the same sum of biases tie, whatever the roundings
                    bad = nan[t, v[0]] or nan[t, v[1]]
                    top.append(-np.inf if bad else (s[t, v[0]] + s[t, v[1]]) + (bias[v[0]] + bias[v[1]]))
                else:
                    top.append(c[t, v[0]])
            kept = sorted(range(n_group), key=lambda g: (-top[g], g))[:topk_group]
            allowed = [e for e in range(E) if e // gs in kept]
        ids[t] = sorted(allowed, key=lambda e: (-c[t, e], e))[:k]
    raw = np.take_along_axis(logits, ids.astype(np.int64), 1)
    w = np.take_along_axis(s, ids.astype(np.int64), 1)
    if renormalize:
        num = ~np.isnan(raw)
        l = _finite(np.where(num, raw, 0.0))
        # relative to the largest chosen log score, so that scores below the smallest number
        # of the format keep their ratios
        ls = l if score == "softmax" else np.where(l > -700, -np.logaddexp(0.0, -np.maximum(l, -700)), l)
        m = np.max(np.where(num, ls, -np.inf), axis=1, keepdims=True)
        e = np.where(num, np.exp(np.where(num, ls - np.where(np.isfinite(m), m, 0.0), 0.0)), 0.0)
        tot = e.sum(1, keepdims=True)
        w = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
    return ids, w * scale


def sort_pairs(ids, adapter_ids, E, L):
    """The stable (expert, adapter) order of the pairs and its CSR offsets."""
    M, k = ids.shape
    keys = [int(ids[t, j]) * (L + 1) + (int(adapter_ids[t]) if adapter_ids[t] >= 0 else L)
            for t in range(M) for j in range(k)]
    pairs = sorted(range(M * k), key=lambda p: (keys[p], p))
    count = np.bincount(np.asarray(keys, dtype=np.int64), minlength=E * (L + 1)) if M else np.zeros(E * (L + 1))
    return np.asarray(pairs, dtype=np.int32), np.concatenate([[0], np.cumsum(count)]).astype(np.int32)


def activation(name: str, h: np.ndarray, h_out: int) -> np.ndarray:
    sig = lambda v: np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))
    if name == "none":
        return h
    if name == "relu":
        return np.maximum(h, 0.0)
    if name == "gelu":
        return 0.5 * h * (1 + np.vectorize(math.erf, otypes=[float])(h / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * h * (1 + np.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)))
    if name == "silu":
        return h * sig(h)
    g, u = h[:, :h_out], h[:, h_out:]
    return g * sig(g) * u


def row_adapters(T, seg_offsets, seg_adapter):
    """Adapter of every token; -1 outside all segments."""
    a = np.full(T, -1, dtype=np.int64)
    for s in range(len(seg_adapter)):
        a[seg_offsets[s]:seg_offsets[s + 1]] = seg_adapter[s]
    return a


def dense_fused(x, w, a, b, rows, *, bias=None, act="none", residual=None, lora_scale=1.0):
    """(y, spread): y of the definition, and per element of h what a rounding analysis needs:
    dict(abs=sum |x w|, lora=lora_scale * sum_i |z_i B_i|, h=h)."""
    n = w.shape[0]
    h_out = n // 2 if act == "silu_and_mul" else n
    h = x @ w.T
    mass = np.abs(x) @ np.abs(w).T
    lora = np.zeros_like(h)
    lmass = np.zeros_like(h)
    if a is not None:
        for ad in range(a.shape[0]):
            t = np.flatnonzero(rows == ad)
            if t.size:
                z = x[t] @ a[ad].T
                h[t] += lora_scale * (z @ b[ad])
                lora[t] = abs(lora_scale) * (np.abs(z) @ np.abs(b[ad]))
                lmass[t] = abs(lora_scale) * ((np.abs(x[t]) @ np.abs(a[ad]).T) @ np.abs(b[ad]))
    if bias is not None:
        h = h + bias[None, :]
        mass = mass + np.abs(bias)[None, :]
    y = activation(act, h, h_out)
    out = y if residual is None else y + residual
    return out, dict(h=h, act=y, mass=mass, lora=lora, lmass=lmass)
