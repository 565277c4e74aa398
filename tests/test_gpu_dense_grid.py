"""GPU parity of dense_lora_fused on inputs whose sums are exact: nothing but the output's
rounding and the activation's evaluation is allowed for, so that a K block, a rank step or a
group of adapters that is lost or taken twice shows at every depth."""
import pytest
import torch

from tests.fused_cases import run_dense
from tests.grid_cases import SIZES, check_grid, grid_inputs

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
