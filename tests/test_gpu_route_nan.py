"""moe_lora_route_scored where an expert's logit and its bias are both NaN."""
import numpy as np
import pytest
import torch

import moe_lora_b200 as ml
from tests.fused_cases import adapters, check_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E", [(3, 24), (40, 100), (300, 200)])
def test_nan_logit_and_nan_bias_of_one_expert(M, E, score, renormalize):
    """Its weight is 0 and it has no share in the others' softmax, in rows masked but for it too."""
    g = np.random.default_rng(M)
    lg = g.standard_normal((M, E)).astype(np.float32)
    lg[0] = -np.inf
    lg[1, 1:] = -np.inf
    lg[2, 4:] = np.finfo(np.float32).min
    lg[:, 3] = np.nan
    b = (g.standard_normal(E) * 0.05).astype(np.float32)
    b[[3, 7]] = np.nan
    ad = adapters(M, 2, 1)
    for fmt in (dict(), dict(n_group=4, topk_group=2, group_rule="max")):
        fmt = dict(score=score, renormalize=renormalize, **fmt)
        res = ml.route_scored(torch.from_numpy(ad).cuda(), 4, 2, logits_in=torch.from_numpy(lg).cuda(),
                              score_bias=torch.from_numpy(b).cuda(), **fmt)
        torch.cuda.synchronize()
        check_route(res, lg.astype(np.float64), ad, E, 4, 2, score_bias=b.astype(np.float64), **fmt)
        with pytest.raises(ml.MoELoRAError) as ei:
            ml.check_status(res["workspace"])
        assert ei.value.status == ml.ERR_DEVICE_CHECK
