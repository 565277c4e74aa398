"""The status word of dense_lora_fused where there is little to do."""
import pytest
import torch

import moe_lora_b200 as ml
from tests.fused_cases import check_dense, dense_inputs, dev, run_dense

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L", [0, 3])
def test_a_call_without_tokens_clears_it(L):
    d = dense_inputs(9, 72, 136, 3, 8, torch.bfloat16, "none", True, False, 1)
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, 9, 72, 136, 1, 1, 3, 8), "cuda")
    bad = dict(d, offs=torch.tensor([0, 9], dtype=torch.int32), segs=torch.tensor([7], dtype=torch.int32))
    q = {k: dev(v) for k, v in d.items()}
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    lora = (q["a"], q["b"], none, none[:0]) if L else ()

    def empty():
        y = ml.dense_lora_fused(q["x"][:0], q["w"], *lora, bias=q["bias"], workspace=ws)
        assert y.shape == (0, 136)

    run_dense(bad, workspace=ws)  # leaves a device check behind
    empty()
    ml.check_status(ws)
    ws.fill_(171)  # a workspace as torch.empty may give it
    empty()
    ml.check_status(ws)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [9, 300])
def test_segments_without_adapters_are_not_looked_at(T, dt):
    d = dense_inputs(T, 72, 136, 0, 0, dt, "silu", True, True, 1)
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, T, 72, 136, 1, 1, 0, 0), "cuda")
    d["offs"], d["segs"] = torch.tensor([5, -3, T + 9], dtype=torch.int32), torch.tensor([4, -7], dtype=torch.int32)
    y = run_dense(d, workspace=ws)
    ml.check_status(ws)
    check_dense(dict(d, segs=None), y)
