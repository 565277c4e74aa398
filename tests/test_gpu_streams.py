"""Calls of scored routing and the fused projection on a stream that is not the current one, with
work queued on the current one."""
import numpy as np
import pytest
import torch

import moe_lora_b200 as ml
from tests.fused_cases import adapters, check_dense, check_route, dense_inputs, dev

pytestmark = pytest.mark.gpu
PAUSE = 20_000_000  # cycles, about 10 ms


def _queued_reader(n, dtype):
    """A block that a queued copy has yet to read, freed: (the copy, what it has to hold)."""
    src = torch.arange(n, device="cuda").to(dtype)
    want, got = src.clone(), torch.empty_like(src)
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    got.copy_(src)
    return got, want  # src is free now, its reader still waits


@pytest.mark.parametrize("T", [40, 300])
def test_outputs_do_not_take_a_block_that_is_still_read(T):
    d = dense_inputs(T, 264, 512, 3, 16, torch.bfloat16, "silu", True, True, T)
    q = {k: dev(v) for k, v in d.items()}
    lg = torch.from_numpy(np.random.default_rng(T).standard_normal((T, 64)).astype(np.float32)).cuda()
    ad = adapters(T, 3, 1)
    ids = torch.from_numpy(ad).cuda()
    side = torch.cuda.Stream()
    dense = lambda: ml.dense_lora_fused(q["x"], q["w"], q["a"], q["b"], q["offs"], q["segs"], bias=q["bias"],
                                        activation="silu", residual=q["residual"], lora_scale=0.5, stream=side)
    route = lambda: ml.route_scored(ids, 4, 3, logits_in=lg, score="sigmoid", stream=side)
    dense(), route()
    torch.cuda.synchronize()
    sizes = [T * 512 // 2, ml.workspace_size(ml.OP_DENSE_FUSED, T, 264, 512, 1, 1, 3, 16) // 4, 4 * T, 2048]
    for _ in range(3):
        for n in sizes:
            got, want = _queued_reader(n, torch.int32)
            y = dense()
            rt = route()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
            check_dense(d, y)
            check_route(rt, lg.double().cpu().numpy(), ad, 64, 4, 3, score="sigmoid")


def test_outputs_outlive_work_on_the_current_stream():
    """An output read by queued work of the current stream and dropped: the next call on the side
    stream does not write over it."""
    T = 64
    d = dense_inputs(T, 264, 512, 0, 0, torch.bfloat16, "none", True, False, 1)
    q = {k: dev(v) for k, v in d.items()}
    other = q["x"] * 3
    side = torch.cuda.Stream()
    call = lambda x: ml.dense_lora_fused(x, q["w"], bias=q["bias"], stream=side)
    call(other)
    want = call(q["x"])
    torch.cuda.synchronize()
    want = want.clone()
    for _ in range(3):
        y = call(q["x"])
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(PAUSE)
        got = y.clone()
        del y
        call(other)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_captured_on_a_given_stream():
    d = dense_inputs(30, 264, 136, 2, 8, torch.bfloat16, "gelu", True, True, 1)
    q = {k: dev(v) for k, v in d.items()}
    side = torch.cuda.Stream()
    call = lambda: ml.dense_lora_fused(q["x"], q["w"], q["a"], q["b"], q["offs"], q["segs"], bias=q["bias"],
                                       activation="gelu", residual=q["residual"], lora_scale=0.5, stream=side)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y = call()
    y.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    check_dense(d, y)
