"""Pins of the oracle's scored routing and fused projection: torch routines, closed forms and
the plain routing it extends."""
import numpy as np
import pytest
import torch

from oracle import fused_ref as fr
from oracle import moe_lora_ref as ref


def _lg(M, E, seed):
    return np.random.default_rng(seed).standard_normal((M, E)).astype(np.float32).astype(np.float64)


def test_defaults_are_the_plain_routing():
    lg = _lg(40, 24, 1)
    ids, w = fr.route_scored(lg, 6)
    ids0, w0 = ref.route_topk(lg, 6)
    assert np.array_equal(ids, ids0)
    np.testing.assert_allclose(w, w0, rtol=1e-12)
    ad = np.random.default_rng(2).integers(-1, 3, 40)
    for got, want in zip(fr.sort_pairs(ids, ad, 24, 3), ref.sort_pairs(ids0, ad, 24, 3)):
        assert np.array_equal(got, want)


def test_scores_are_torch_scores():
    lg = _lg(9, 30, 3)
    t = torch.from_numpy(lg)
    np.testing.assert_allclose(fr.scores(lg, "softmax"), torch.softmax(t, 1).numpy(), rtol=1e-12)
    np.testing.assert_allclose(fr.scores(lg, "sigmoid"), torch.sigmoid(t).numpy(), rtol=1e-12)


def test_bias_moves_the_choice_not_the_weight():
    lg = np.zeros((1, 4))
    ids, w = fr.route_scored(lg, 2, score="sigmoid", score_bias=np.array([0.0, 0.2, 0.0, 0.1]), renormalize=False,
                             scale=3.0)
    assert ids.tolist() == [[1, 3]] and w.tolist() == [[1.5, 1.5]]


@pytest.mark.parametrize("rule,want", [("max", [5, 4]), ("top2", [1, 0])])
def test_group_rules(rule, want):
    lg = np.array([[2.0, 2.1, 0.0, 0.0, 1.0, 2.2]])  # groups of two
    ids, _ = fr.route_scored(lg, 2, score="sigmoid", n_group=3, topk_group=1, group_rule=rule)
    assert ids.tolist() == [want]


def test_masked_and_nan_rows():
    inf, nan = np.inf, np.nan
    lg = np.array([[-inf, 1.0, -inf, nan], [-inf] * 4, [nan] * 4])
    ids, w = fr.route_scored(lg, 2, score="sigmoid")
    assert ids.tolist() == [[1, 0], [0, 1], [0, 1]]
    np.testing.assert_allclose(w, [[1, 0], [0.5, 0.5], [0, 0]], atol=1e-300)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "silu_and_mul"])
def test_projection_against_torch(act):
    g = np.random.default_rng(5)
    x, w, b = g.standard_normal((7, 16)), g.standard_normal((24, 16)), g.standard_normal(24)
    y, _ = fr.dense_fused(x, w, None, None, np.full(7, -1), bias=b, act=act)
    h = torch.nn.functional.linear(*(torch.from_numpy(v) for v in (x, w, b)))
    F = torch.nn.functional
    want = {"none": h, "relu": F.relu(h), "gelu": F.gelu(h), "gelu_tanh": F.gelu(h, approximate="tanh"),
            "silu": F.silu(h), "silu_and_mul": F.silu(h[:, :12]) * h[:, 12:]}[act]
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-10, atol=1e-12)


def test_projection_adapters_against_the_plain_projection():
    g = np.random.default_rng(6)
    x, w = g.standard_normal((9, 8)), g.standard_normal((6, 8))
    a, b = g.standard_normal((2, 3, 8)), g.standard_normal((2, 3, 6))
    offs, segs = np.array([0, 4, 6, 9]), np.array([1, -1, 0])
    rows = fr.row_adapters(9, offs, segs)
    assert rows.tolist() == [1] * 4 + [-1] * 2 + [0] * 3
    res = g.standard_normal((9, 6))
    y, _ = fr.dense_fused(x, w, a, b, rows, residual=res, lora_scale=1.0)
    np.testing.assert_allclose(y, ref.dense_lora_forward(x, w, a, b, offs, segs) + res, rtol=1e-12)
