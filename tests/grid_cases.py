"""Inputs of the fused dense projection whose sums are exact in fp32, and tolerances that count
roundings alone.

A bound that grows with the length of a sum cannot see a lost block of a long one.  Here x, W, A,
B, bias and residual are small integers times powers of two, so that every partial sum of
h = x W^T + bias + c (x A) B, in any order, is a whole number of steps below 2^24: fp32 holds it
exactly, and so do two bf16 numbers z = c x A (at most 2^16 steps; asserted).  What is left of an
error is the activation's evaluation and one rounding to the output's type.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import fused_ref as fr
from tests.fused_cases import dense_oracle, segments

SCALE = 0.5


def _ints(g, shape, std, most):
    return np.clip(np.round(g.standard_normal(shape) * std), -most, most)


def _bits(n):
    """b with 2 * 2^-b near n^-0.5: the deviation of two steps."""
    return int(round(np.log2(2.0 * np.sqrt(n))))


def grid_inputs(T, h_in, h_out, L, r, dt, act, bias, residual, seed, none_frac=0.2, grouped=True):
    """The dict of fused_cases.dense_inputs, on grids."""
    g = np.random.default_rng(seed)
    n = 2 * h_out if act == "silu_and_mul" else h_out

    def t(v):
        q = torch.from_numpy(v).to(dt)
        assert np.array_equal(q.double().numpy(), v)  # the type holds every one of them
        return q

    bw, br = _bits(h_in), _bits(r) if L else 0
    zstep = 2.0 ** -(2 + bw + 1 + 1)  # of c x A; x W^T has four times that
    step = zstep * 2.0 ** -br if L else 4 * zstep  # of every sum (bias and residual: 1/8)
    x, w = _ints(g, (T, h_in), 4.0, 15) / 4, _ints(g, (n, h_in), 2.0, 7) * 2.0 ** -bw
    mass = np.abs(x) @ np.abs(w).T
    d = dict(x=t(x), w=t(w), a=None, b=None, offs=None, segs=None, bias=None, residual=None, act=act, scale=SCALE)
    if bias:
        b = _ints(g, (n,), 4.0, 15) / 8
        d["bias"], mass = t(b), mass + np.abs(b)
    if residual:
        d["residual"] = t(_ints(g, (T, h_out), 8.0, 31) / 8)
    if L > 0:
        a = _ints(g, (L, r, h_in), 4.0, 15) * 2.0 ** -(bw + 1)
        b = _ints(g, (L, r, n), 2.0, 7) * 2.0 ** -br
        d["a"], d["b"] = t(a), t(b)
        offs, segs = segments(T, L, seed + 1, none_frac, grouped)
        d["offs"], d["segs"] = torch.from_numpy(offs), torch.from_numpy(segs)
        rows = fr.row_adapters(T, offs, segs)
        for ad in range(L):
            i = np.flatnonzero(rows == ad)
            if i.size:
                z = SCALE * (x[i] @ a[ad].T)
                assert np.abs(z).max() <= 2.0 ** 16 * zstep
                mass[i] += np.abs(z) @ np.abs(b[ad])
    assert T == 0 or mass.max() < 2.0 ** 24 * min(step, 0.125)
    return d


def spacing(v, dt):
    """Distance of neighbouring numbers of the type around |v| (normal numbers)."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126)))
    return 2.0 ** (e - (7 if dt == torch.bfloat16 else 23))


def grid_tolerance(d, y, m):
    """Largest |error| of each element of y.

    h: exact.  act: none and relu exact; the others within 2^-20 of the result in fp32 (expf, erff
    and tanh forms, a quotient and a product, each within a few 2^-23), plus 2^-22 |h| where
    1 + erf or 1 + tanh cancels; a gated product adds 2^-23.  The fast exponential of bf16 outputs
    is off by 2 + 1.173 |x| units of at most 2^-23: 2^-22 |x| on top, x = h or 1.6 (h + 0.045 h^3).  The residual's add in fp32: half a
    step of 2^-23.  y: half of its type's spacing."""
    dt = d["x"].dtype
    h = m["h"][:, : y.shape[1]]
    ea = np.zeros_like(y)
    if d["act"] not in ("none", "relu"):
        rel = 2.0 ** -20
        if dt == torch.bfloat16 and d["act"] != "gelu":
            rel = rel + 2.0 ** -22 * np.abs(1.6 * (h + 0.045 * h ** 3) if d["act"] == "gelu_tanh" else h)
        ea = rel * np.abs(m["act"]) + (2.0 ** -22 * np.abs(h) if d["act"].startswith("gelu") else 0.0)
    if d["residual"] is not None and d["act"] not in ("none", "relu"):
        ea = ea + 2.0 ** -24 * np.abs(y)
    return ea + 0.5 * spacing(np.abs(y) + ea, dt)


def grid_error(d, got, rows=None):
    """Largest error of `got` (an array or tensor [T, h_out]) in units of its tolerance."""
    y, m = dense_oracle(d, rows)
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    return float(np.max(np.abs(got - y) / grid_tolerance(d, y, m))) if y.size else 0.0


def check_grid(d, got, rows=None):
    worst = grid_error(d, got, rows)
    assert worst <= 1.0, f"error {worst:.2f} of the tolerance"


# sizes by the form that they take: up to 16, 32, 64, 128 and 256 tokens with the shrink on CUDA
# cores or the tensor cores; a split reduction above 256; tiles of 256 x 256.  K blocks (64) even
# over the splits, uneven, a last one of 8; adapters' groups fewer and more than the K blocks.
SIZES = [(1, 4104, 264, 6, 16), (1, 11008, 136, 6, 128), (4, 2056, 264, 5, 16), (16, 520, 200, 4, 8), (31, 1032, 264, 7, 32),
         (64, 4096, 520, 22, 16), (64, 11008, 136, 5, 64), (65, 1032, 392, 9, 8), (128, 72, 136, 3, 128),
         (203, 2056, 1000, 5, 8), (256, 776, 264, 12, 64), (300, 2048, 264, 6, 32), (520, 4104, 136, 20, 8),
         (300, 264, 520, 7, 16), (700, 328, 264, 9, 64), (1100, 200, 520, 33, 8), (900, 264, 264, 5, 128)]

# a token or a few, over every split of the reduction
FEW = [(T, h_in, h_out, 6, r) for T, r in [(1, 8), (1, 16), (2, 8), (1, 32), (1, 128), (2, 16), (3, 8), (4, 16)]
       for h_in, h_out in [(8, 8), (72, 200), (4104, 1000), (11008, 264)]]
# token counts on both sides of every tile width; K and features that end inside a block
EDGES = [(T, h_in, h_out, 5, 16) for T, h_in, h_out in
         [(1, 8, 8), (2, 72, 8), (8, 4096, 512), (16, 512, 520), (17, 2056, 264), (32, 1024, 1000), (33, 64, 136),
          (64, 2048, 1408), (65, 520, 392), (127, 128, 128), (128, 1032, 640), (129, 256, 264), (200, 776, 1000),
          (255, 64, 512), (256, 2048, 256), (257, 264, 520), (384, 1000, 776), (511, 512, 512), (640, 200, 1032),
          (1025, 328, 264)]]
