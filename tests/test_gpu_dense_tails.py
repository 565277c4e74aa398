"""The activations of dense_lora_fused over the whole range of h: where exp overflows, where the
result is small, at signed zeros and beyond the largest finite number."""
import math

import numpy as np
import pytest
import torch

import moe_lora_b200 as ml
from oracle import fused_ref as fr
from tests.grid_cases import spacing

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
N = 8


def _through(values, act, dt, up=None):
    """act(h) of h = the values, exactly: h_in = 8, a token's x is (value, up, 0, ...)."""
    x = torch.zeros((len(values), 8), dtype=dt)
    x[:, 0] = torch.tensor(values, dtype=dt)
    w = torch.zeros((2 * N if act == "silu_and_mul" else N, 8), dtype=dt)
    w[:N, 0] = 1
    if act == "silu_and_mul":
        x[:, 1] = torch.tensor(up, dtype=dt)
        w[N:, 1] = 1
    y = ml.dense_lora_fused(x.cuda(), w.cuda(), activation=act).double().cpu().numpy()
    assert np.array_equal(y, np.repeat(y[:, :1], N, 1), equal_nan=True)
    return x[:, 0].double().numpy(), y[:, 0]


def _exact(act, h):
    if act == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)
        return h * np.where(u > 0, 1 / (1 + np.exp(-np.abs(u))), np.exp(-np.abs(u)) / (1 + np.exp(-np.abs(u)))), np.abs(u)
    return fr.activation("silu", h, h.size), np.abs(h)


# every count of tokens takes another form of the kernel
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("copies", [1, 4, 40])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "silu_and_mul"])
def test_small_results(act, copies, dt):
    """silu and the tanh GELU of -104 to 104.  Their exponential is off by 2 units of the last place
    (bf16: 2 + 1.173 |x|, under 2^-22 + |x| 2^-22) and its argument by 4 roundings (2^-22 of it), the
    sum, quotient and product by 2^-22; below the smallest normal number the exponential is off by 2
    steps of 2^-149, times |h|."""
    values = [float(v) for v in np.arange(-104, 104.5, 0.5)]
    if act == "gelu_tanh":
        values = [v / 8 for v in values]
    up = [0.125] * (len(values) * copies)
    h, y = _through(values * copies, act, dt, up)
    want, arg = _exact(act, h)
    tol = (2.0 ** -20 + 2.0 ** -21 * arg) * np.abs(want) + 2.0 ** -148 * np.abs(h)
    if act == "silu_and_mul":
        want, tol = want / 8, tol / 8 + 2.0 ** -149
    tol = tol + 0.5 * spacing(np.abs(want) + tol, dt)
    worst = np.argmax(np.abs(y - want) / tol)
    assert np.abs(y - want)[worst] <= tol[worst], f"act({h[worst]}) = {y[worst]}, not {want[worst]}"


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T", [8, 300])
def test_ends(T, dt):
    """Infinities, NaN, zeros and the largest numbers through every activation."""
    big = float(torch.finfo(torch.bfloat16).max)
    values = [float("nan"), float("inf"), 0.0, -0.0, big, -big, 1e20, -1e20] * (T // 8)
    for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
        h, y = _through(values, act, dt)
        y = y.reshape(-1, 8)
        assert np.isnan(y[:, 0]).all() and np.isposinf(y[:, 1]).all() and (y[:, 2:4] == 0).all()
        assert (y[:, [4, 6]] == h.reshape(-1, 8)[:, [4, 6]]).all()
        assert (y[:, [5, 7]] == (h.reshape(-1, 8)[:, [5, 7]] if act == "none" else 0)).all()
