"""GPU parity of dense_lora_fused on inputs whose sums are exact: nothing but the output's
rounding and the activation's evaluation is allowed for, so that a K block, a rank step or a
group of adapters that is lost or taken twice shows at every depth."""
import numpy as np
import pytest
import torch

from oracle import fused_ref as fr
from tests.fused_cases import dense_oracle, run_dense
from tests.grid_cases import EDGES, FEW, SIZES, check_grid, grid_inputs, grid_tolerance

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("act", ["none", "silu_and_mul"])
@pytest.mark.parametrize("T,h_in,h_out,L,r", SIZES)
def test_sums_are_exact(T, h_in, h_out, L, r, act):
    for kw in (dict(), dict(grouped=False, none_frac=0.0)):
        d = grid_inputs(T, h_in, h_out, L, r, BF16, act, True, True, T + h_in, **kw)
        check_grid(d, run_dense(d))
    d = grid_inputs(T, h_in, h_out, 0, 0, BF16, act, True, False, T + h_in + 1)
    check_grid(d, run_dense(d))


@pytest.mark.parametrize("act", ["none", "silu_and_mul"])
@pytest.mark.parametrize("T,h_in,h_out,L,r", FEW + EDGES)
def test_sums_are_exact_at_the_edges(T, h_in, h_out, L, r, act):
    d = grid_inputs(T, h_in, h_out, L, r, BF16, act, True, True, T + h_in, none_frac=0.0, grouped=T > 4)
    check_grid(d, run_dense(d))


@pytest.mark.parametrize("act", ["none", "silu_and_mul"])
@pytest.mark.parametrize("T,h_in,h_out,L,r", [(1, 520, 264, 3, 16), (19, 2048, 136, 4, 8), (64, 512, 512, 4, 16),
                                              (200, 1576, 264, 3, 128), (512, 2048, 264, 2, 64)])
def test_sums_are_exact_f32(T, h_in, h_out, L, r, act):
    for kw in (dict(), dict(grouped=False, none_frac=0.0)):
        d = grid_inputs(T, h_in, h_out, L, r, F32, act, True, True, T + h_in, **kw)
        check_grid(d, run_dense(d))
    d = grid_inputs(T, h_in, h_out, 0, 0, F32, act, True, False, T + h_in + 1)
    check_grid(d, run_dense(d))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T,h_in,h_out,L,r", [(40, 1032, 264, 4, 16), (300, 264, 264, 4, 16), (300, 2048, 264, 4, 16)])
def test_activations(T, h_in, h_out, L, r, act):
    for dt in (BF16, F32):
        d = grid_inputs(T, h_in, h_out, L, r, dt, act, True, True, T)
        check_grid(d, run_dense(d))


@pytest.mark.parametrize("act", ["none", "silu_and_mul"])
@pytest.mark.parametrize("T,h_in,h_out", [(261, 264, 520), (700, 264, 136), (300, 2048, 136), (45, 520, 264)])
def test_lanes_of_a_warp_that_part(T, h_in, h_out, act):
    """Neighbouring tokens with adapters of their own, every third one broken or none at all, and
    rows that end inside a warp: threads that take other turns join again ahead of each collective
    instruction."""
    d = grid_inputs(T, h_in, h_out, 9, 16, BF16, act, True, True, T, grouped=False)
    rows = fr.row_adapters(T, d["offs"].numpy(), d["segs"].numpy())
    b = d["b"].clone()
    for ad in (1, 4, 7):
        b[ad, ad, 5] = float("inf")
    y = run_dense({**d, "b": b}).cpu()
    clean = torch.ones(h_out, dtype=torch.bool)
    clean[5] = False
    broken = torch.from_numpy(np.isin(rows, (1, 4, 7)))
    assert not torch.isfinite(y[broken, 5]).any() and torch.isfinite(y[~broken]).all()
    want, m = dense_oracle(d)
    off = np.abs(y.double().numpy() - want) / grid_tolerance(d, want, m)
    assert off[~broken.numpy()].max() <= 1.0 and off[:, clean.numpy()].max() <= 1.0
