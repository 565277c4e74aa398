"""Builders for the tests of scored routing and the fused dense projection (GPU against the
fp64 oracle), with the tolerances derived here."""
from __future__ import annotations

import numpy as np
import torch

import moe_lora_b200 as ml
from oracle import fused_ref as fr


def adapters(M, L, seed, none_frac=0.2):
    g = np.random.default_rng(seed)
    a = g.integers(0, max(L, 1), size=M).astype(np.int32)
    a[(g.random(M) < none_frac) | (L == 0)] = -1
    return a


def check_route(res, logits64, ad, E, k, L, **fmt):
    """ids, pairs and offsets equal the oracle's; weights within fp32 rounding.

    A weight is a quotient of expf results and a sum of at most 256 of them: each expf is off
    by at most 2 ulp (2^-22) plus the rounding of its argument (|l - top| 2^-24, under 2^-17
    for the |l| < 100 the tests use), the sum by 8 + 8 roundings (lanes, then the warp), two
    quotients by 2^-24 each: under 2^-16 relative in all."""
    ids, w = fr.route_scored(logits64, k, **fmt)
    sp, so = fr.sort_pairs(ids, ad, E, L)
    assert np.array_equal(res["topk_ids"].cpu().numpy(), ids)
    np.testing.assert_allclose(res["topk_w"].cpu().numpy(), w, rtol=2.0 ** -16, atol=1e-37)
    assert np.array_equal(res["sorted_pairs"].cpu().numpy(), sp)
    assert np.array_equal(res["seg_offsets"].cpu().numpy(), so)


def grid_router(M, E, H, seed):
    """x and W_r on grids (1/16 and a power of two near 1/16 of W_r's deviation): every
    partial sum of a logit is a multiple of the product grid below 2^24 of its steps, so fp32
    sums are exact in any order and the logits of every kernel equal the fp64 ones."""
    g = np.random.default_rng(seed)
    x = np.clip(np.round(g.standard_normal((M, H)) * 16), -64, 64) / 16
    bits = int(np.ceil(np.log2(16 * np.sqrt(H))))
    w = np.clip(np.round(g.standard_normal((E, H)) / np.sqrt(H) * 2.0 ** bits), -64, 64) * 2.0 ** -bits
    lg = x @ w.T
    assert M == 0 or np.max(np.abs(x) @ np.abs(w).T) * 2.0 ** (bits + 4) < 2.0 ** 24
    return torch.from_numpy(x).to(torch.bfloat16), torch.from_numpy(w).to(torch.bfloat16), lg


def segments(T, L, seed, none_frac=0.2, grouped=True):
    """(offsets, adapters) of maximal runs: tokens grouped by adapter, or in arrival order."""
    ids = adapters(T, L, seed, none_frac)
    if grouped:
        ids = np.sort(ids)
    starts = [0] + [i for i in range(1, T) if ids[i] != ids[i - 1]]
    return np.array(starts + [T], dtype=np.int32), ids[starts].astype(np.int32)


def dense_inputs(T, h_in, h_out, L, r, dt, act, bias, residual, seed, none_frac=0.2, grouped=True):
    g = torch.Generator().manual_seed(seed)
    n = 2 * h_out if act == "silu_and_mul" else h_out
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt)
    d = dict(x=rnd(T, h_in), w=rnd(n, h_in, std=h_in ** -0.5), a=None, b=None, offs=None, segs=None,
             bias=rnd(n, std=0.5) if bias else None, residual=rnd(T, h_out) if residual else None, act=act, scale=0.5)
    if L > 0:
        d["a"], d["b"] = rnd(L, r, h_in, std=h_in ** -0.5), rnd(L, r, n, std=r ** -0.5)
        offs, segs = segments(T, L, seed + 1, none_frac, grouped)
        d["offs"], d["segs"] = torch.from_numpy(offs), torch.from_numpy(segs)
    return d


def dev(v):
    return v.cuda() if isinstance(v, torch.Tensor) else v


def run_dense(d, **kw):
    q = {k: dev(v) for k, v in d.items()}
    return ml.dense_lora_fused(q["x"], q["w"], q["a"], q["b"], q["offs"], q["segs"], bias=q["bias"],
                               activation=d["act"], residual=q["residual"], lora_scale=d["scale"], **kw)


def dense_oracle(d, rows=None):
    f = lambda t: None if t is None else t.double().numpy()
    T = d["x"].shape[0]
    if rows is None:
        rows = np.full(T, -1) if d["segs"] is None else fr.row_adapters(T, d["offs"].numpy(), d["segs"].numpy())
    return fr.dense_fused(f(d["x"]), f(d["w"]), f(d["a"]), f(d["b"]), rows, bias=f(d["bias"]), act=d["act"],
                          residual=f(d["residual"]), lora_scale=d["scale"])


def dense_tolerance(d, y, m):
    """Largest |error| of each element of y.

    h: a sum of K products in fp32 is off by at most K u of its mass, u = 2^-24 for rounded
    adds and 2^-23 where the tensor core truncates; xA likewise, carried through B.  bf16
    rounds z = c xA once: half a step, 2^-8 of each z_i.
    act: slopes are at most 1.13 (gelu, tanh gelu and silu; the largest is gelu's 1.129), and
    2^-18 of the result covers the fp32 evaluation (erff, tanhf, expf within 4 ulp, their
    argument's and the product's roundings), with 2^-18 |h| where 1 + erf or 1 + tanh cancels.
    A gated product: each factor's error times the other factor.
    y: half a step of its type, and one rounding of the residual's add in fp32."""
    bf16 = d["x"].dtype == torch.bfloat16
    K = d["x"].shape[1] + (d["a"].shape[1] if d["a"] is not None else 0) + 2
    u = 2.0 ** -23 if bf16 else 2.0 ** -24
    eh = K * u * (m["mass"] + m["lmass"]) + (2.0 ** -8 * m["lora"] if bf16 else 0.0)
    if d["act"] == "silu_and_mul":
        n = y.shape[1]
        g, up = m["h"][:, :n], m["h"][:, n:]
        sg = fr.activation("silu", g, n)
        ea = 1.13 * eh[:, :n] * (np.abs(up) + eh[:, n:]) + np.abs(sg) * eh[:, n:] + 2.0 ** -18 * np.abs(sg * up)
    elif d["act"] in ("none", "relu"):
        ea = eh
    else:
        ea = 1.13 * eh + 2.0 ** -18 * np.abs(m["h"])
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    return half * (np.abs(y) + ea) + ea + 2.0 ** -23 * (np.abs(y) + np.abs(m["act"]))


def check_dense(d, got, rows=None, where=None):
    y, m = dense_oracle(d, rows)
    tol = dense_tolerance(d, y, m)
    err = np.abs(got.detach().float().cpu().numpy().astype(np.float64) - y)
    if where is not None:
        err, tol = err[where], tol[where]
    worst = float(np.max(err / tol)) if err.size else 0.0
    assert worst <= 1.0, f"error {worst:.2f} of the tolerance at {np.unravel_index(np.argmax(err / tol), err.shape)}"
