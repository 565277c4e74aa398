"""Host-side refusals of moe_lora_route_scored and dense_lora_fused: every call below fails
validation before anything is launched (the fake addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import moe_lora_b200 as ml

FAKE = 0x7F0000000000
MIS = FAKE + 4
INV, UNS = ml.ERR_INVALID_ARG, ml.ERR_UNSUPPORTED


def _route(fmt=(1, 1, 1, 0, 1, 1.0), **kw):
    a = dict(x=FAKE, wr=FAKE, bias=None, lin=None, sb=None, ad=FAKE, M=4, H=64, E=8, k=2, L=2, lout=None, ids=FAKE,
             w=FAKE, sp=FAKE, so=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    f = None if fmt is None else ctypes.byref(ml.RouteFormat(*fmt))
    return ml.lib().moe_lora_route_scored(a["x"], a["wr"], a["bias"], a["lin"], a["sb"], a["ad"], a["M"], a["H"],
                                          a["E"], a["k"], a["L"], f, a["lout"], a["ids"], a["w"], a["sp"], a["so"],
                                          a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fmt,code", [
    ((2, 1, 1, 0, 1, 1.0), INV), ((-1, 1, 1, 0, 1, 1.0), INV),      # score
    ((1, 0, 1, 0, 1, 1.0), INV), ((1, 3, 1, 0, 1, 1.0), INV),       # n_group does not divide E
    ((1, 16, 1, 0, 1, 1.0), INV), ((1, 4, 5, 0, 1, 1.0), INV),      # more groups than there are
    ((1, 4, 0, 0, 1, 1.0), INV), ((1, 8, 1, 0, 1, 1.0), INV),       # the kept groups hold fewer than k
    ((1, 4, 2, 2, 1, 1.0), INV), ((1, 4, 2, 0, 2, 1.0), INV),
    ((1, 1, 1, 0, 1, float("nan")), INV), ((1, 1, 1, 0, 1, float("inf")), INV),
])
def test_route_formats_refused(fmt, code):
    assert _route(fmt) == code
    assert ml.lib().moe_lora_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(so=None), INV), (dict(ad=None), INV), (dict(x=None), INV), (dict(wr=None), INV), (dict(ids=None), INV),
    (dict(sb=MIS), INV), (dict(bias=MIS), INV), (dict(lout=MIS), INV), (dict(lin=MIS), INV), (dict(ws=None), INV),
    (dict(ws=MIS), INV), (dict(wsb=8), INV), (dict(M=-1), INV), (dict(k=0), INV), (dict(k=9), UNS),
    (dict(E=300), UNS), (dict(L=65), UNS), (dict(H=12), UNS), (dict(H=0), UNS), (dict(M=1 << 20, k=2), UNS),
])
def test_route_arguments_refused(kw, code):
    assert _route(**kw) == code
    assert _route(None, **kw) == code


def _dense(**kw):
    a = dict(x=FAKE, w=FAKE, bias=None, A=FAKE, B=FAKE, seg=FAKE, sad=FAKE, S=1, T=8, h_in=64, h_out=64, r=16, L=2,
             act=0, scale=1.0, res=None, dt=ml.ML_BF16, y=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return ml.lib().dense_lora_fused(a["x"], a["w"], a["bias"], a["A"], a["B"], a["seg"], a["sad"], a["S"], a["T"],
                                     a["h_in"], a["h_out"], a["r"], a["L"], a["act"], a["scale"], a["res"], a["dt"],
                                     a["y"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), INV), (dict(x=MIS), INV), (dict(w=None), INV), (dict(bias=MIS), INV), (dict(res=MIS), INV),
    (dict(A=None), INV), (dict(B=None), INV), (dict(seg=None), INV), (dict(sad=None), INV), (dict(S=0), INV),
    (dict(act=6), INV), (dict(act=-1), INV), (dict(dt=ml.ML_E4M3), INV), (dict(T=-1), INV), (dict(h_in=0), INV),
    (dict(h_in=12), UNS), (dict(h_out=20), UNS), (dict(r=24), UNS), (dict(L=65), UNS), (dict(T=(1 << 20) + 1), UNS),
    (dict(h_out=(1 << 20) + 8), UNS), (dict(ws=None), INV), (dict(wsb=10), INV), (dict(ws=MIS), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
])
def test_dense_arguments_refused(kw, code):
    assert _dense(**kw) == code
    assert ml.lib().moe_lora_last_error()


def test_dense_no_tokens_is_ok():
    assert _dense(T=0, S=0, x=None, w=None, y=None, A=None, B=None, seg=None, sad=None) == ml.OK


def test_workspace_sizes():
    assert ml.workspace_size(ml.OP_ROUTE_SCORED, 1000, 0, 0, 64, 8, 8, 0) >= 256 + 64 * 1000 // 8
    assert ml.workspace_size(ml.OP_DENSE_FUSED, 64, 4096, 512, 1, 1, 4, 16) >= 256 + 64 * 16 * 2
    assert ml.workspace_size(ml.OP_DENSE_FUSED, -1) == 0
    # grows with the batch, so a workspace made for the largest batch serves every smaller one
    for op, args in ((ml.OP_ROUTE_SCORED, (1024, 0, 128, 8, 16, 0)), (ml.OP_DENSE_FUSED, (1024, 512, 1, 1, 4, 16))):
        sizes = [ml.workspace_size(op, M, *args) for M in (1, 2, 63, 64, 65, 128, 129, 1000, 2304, 2305, 4096, 9472, 9473)]
        assert sizes == sorted(sizes)


def test_binding_refuses():
    """Wrong types, shapes and words are refused before any device is touched."""
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 32, dtype=torch.bfloat16)
    offs, segs = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    bad = [dict(activation="swish"), dict(bias=torch.zeros(32)), dict(bias=torch.zeros(31, dtype=torch.bfloat16)),
           dict(residual=torch.zeros(4, 31, dtype=torch.bfloat16)), dict(lora_a=a), dict(lora_a=a, lora_b=b),
           dict(lora_a=a, lora_b=b[:, :, :16], seg_offsets=offs, seg_adapter=segs),
           dict(lora_a=a, lora_b=b, seg_offsets=offs.long(), seg_adapter=segs),
           dict(lora_a=a, lora_b=b, seg_offsets=offs[:1], seg_adapter=segs), dict(y=torch.zeros(4, 32))]
    for kw in bad:
        with pytest.raises(ValueError):
            ml.dense_lora_fused(x, w, **kw)
    with pytest.raises(ValueError):
        ml.dense_lora_fused(x.half(), w.half())
    with pytest.raises(ValueError):
        ml.dense_lora_fused(x, w[:31], activation="silu_and_mul")
    with pytest.raises(ValueError):
        ml.dense_lora_fused(x, w.float())
    ad, lg = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8)
    for kw in (dict(logits_in=lg.double()), dict(logits_in=lg, score="tanh"), dict(logits_in=lg, group_rule="sum"),
               dict(logits_in=lg[:3]), dict(), dict(x=x), dict(x=x, w_router=w.float()),
               dict(logits_in=lg, score_bias=torch.zeros(7)), dict(logits_in=lg, out={"topk_w": torch.zeros(3, 2)}),
               dict(logits_in=lg, out={"topk_ids": torch.zeros(4, 2)})):
        with pytest.raises(ValueError):
            ml.route_scored(ad, 2, 2, **kw)
    with pytest.raises(ValueError):
        ml.route_scored(ad.long(), 2, 2, logits_in=lg)
    with pytest.raises(ValueError):  # host tensors
        ml.dense_lora_fused(x, w)
