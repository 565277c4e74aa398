"""dense_lora_fused with more tokens than the operand of the tiled form holds at a time."""
import numpy as np
import pytest
import torch

import moe_lora_b200 as ml
from oracle import fused_ref as fr
from tests.fused_cases import run_dense
from tests.grid_cases import check_grid, grid_inputs

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("T", [8192, 8193, 16384 + 300])
def test_bands_of_tokens(T):
    """64 adapters of rank 128: 8192 tokens at a time.  Broken rows of B and wrong segments anywhere
    are those of the whole call."""
    d = grid_inputs(T, 64, 136, 64, 128, BF16, "silu_and_mul", True, True, T, grouped=False)
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, T, 64, 136, 1, 1, 64, 128), "cuda")
    y = run_dense(d, workspace=ws)
    ml.check_status(ws)
    check_grid(d, y)
    rows = fr.row_adapters(T, d["offs"].numpy(), d["segs"].numpy())
    b = d["b"].clone()
    b[11, 70, 20] = float("nan")
    z = run_dense({**d, "b": b}, workspace=ws)
    ml.check_status(ws)
    mine = torch.from_numpy(rows == 11).cuda()
    assert torch.isnan(z[mine][:, 20]).all() and torch.equal(z[~mine], y[~mine])
    for at in (0, len(d["segs"]) - 1):  # flagged by the first band's tokens, and by the last one's
        segs = d["segs"].clone()
        segs[at] = 64
        bad = rows.copy()
        bad[int(d["offs"][at]):int(d["offs"][at + 1])] = -1
        check_grid(d, run_dense({**d, "segs": segs}, workspace=ws), bad)
        with pytest.raises(ml.MoELoRAError) as ei:
            ml.check_status(ws)
        assert ei.value.status == ml.ERR_DEVICE_CHECK


def test_workspace_is_bounded():
    size = lambda T, L, r: ml.workspace_size(ml.OP_DENSE_FUSED, T, 4096, 4096, 1, 1, L, r)
    assert size(65536, 64, 128) < 320 << 20 and size(1 << 20, 64, 128) < 900 << 20
    assert size(65536, 16, 64) < 320 << 20
