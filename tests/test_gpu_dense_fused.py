"""GPU parity of dense_lora_fused against the fp64 oracle, element by element."""
import numpy as np
import pytest
import torch

import moe_lora_b200 as ml
from oracle import fused_ref as fr
from oracle import moe_lora_ref as ref
from tests.fused_cases import (adapters, check_dense, check_route, dense_inputs, dev, grid_router, run_dense, segments)
from tests.gpu_cases import TOL_BF16, rel_err

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "silu_and_mul"]


def _check(*a, **kw):
    d = dense_inputs(*a, **kw)
    ws_shape = d["x"].shape
    y = run_dense(d)
    torch.cuda.synchronize()
    assert y.shape[0] == ws_shape[0] and y.dtype == d["x"].dtype
    check_dense(d, y)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T", [1, 19, 150, 600])
def test_activations(T, dt, act):
    _check(T, 264, 200, 3, 16, dt, act, True, True, 7 + T)


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("act", ["none", "silu_and_mul"])
@pytest.mark.parametrize("T", [3, 300])
def test_without_bias_or_residual(T, act, bias, residual):
    for dt in (BF16, F32):
        _check(T, 136, 328, 2, 8, dt, act, bias, residual, 5)


# token counts on both sides of every tile width; K and features that end inside a block
SIZES = [(1, 8, 8), (2, 72, 8), (8, 4096, 512), (16, 512, 520), (17, 2056, 264), (32, 1024, 1000), (33, 64, 136),
         (64, 2048, 1408), (65, 520, 392), (127, 128, 128), (128, 1032, 640), (129, 256, 264), (200, 776, 1000),
         (255, 64, 512), (256, 2048, 256), (257, 264, 520), (384, 1000, 776), (511, 512, 512), (640, 200, 1032),
         (1025, 328, 264)]


@pytest.mark.parametrize("act", ["none", "silu_and_mul"])
@pytest.mark.parametrize("T,h_in,h_out", SIZES)
def test_sizes(T, h_in, h_out, act):
    _check(T, h_in, h_out, 5, 16, BF16, act, True, False, T + h_in)
    _check(T, h_in, h_out, 0, 0, BF16, act, False, True, T + h_in + 1)


@pytest.mark.parametrize("T,h_in,h_out", [(1, 8, 8), (5, 520, 136), (64, 512, 512), (65, 72, 200), (300, 264, 328)])
def test_sizes_f32(T, h_in, h_out):
    for act in ("none", "silu_and_mul"):
        _check(T, h_in, h_out, 4, 16, F32, act, True, True, T)
        _check(T, h_in, h_out, 0, 0, F32, act, False, False, T)


@pytest.mark.parametrize("r", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("T", [1, 40, 200, 700])
@pytest.mark.parametrize("act", ["none", "silu_and_mul"])
def test_ranks(T, r, act):
    for dt in (BF16, F32) if T < 700 else (BF16,):
        _check(T, 328, 264, 7, r, dt, act, False, False, r + T)


@pytest.mark.parametrize("T,L", [(64, 64), (64, 1), (300, 64), (300, 33), (1500, 64), (2000, 9)])
def test_many_adapters(T, L):
    _check(T, 256, 392, L, 16, BF16, "gelu", True, True, T + L)
    _check(T, 256, 392, L, 128, BF16, "silu_and_mul", True, True, T + L)


@pytest.mark.parametrize("T", [50, 400, 900])
def test_tokens_in_arrival_order(T):
    """Every maximal run of one adapter is a segment: hundreds of short ones."""
    for L, r in ((4, 64), (20, 8)):
        d = dense_inputs(T, 264, 520, L, r, BF16, "silu", True, True, T, grouped=False)
        assert d["segs"].numel() > T // 3
        check_dense(d, run_dense(d))


def test_no_token_has_an_adapter():
    for T in (20, 500):
        d = dense_inputs(T, 128, 136, 3, 16, BF16, "none", True, False, 1, none_frac=2.0)
        check_dense(d, run_dense(d))


@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_tokens_outside_the_segments(T, dt):
    """A padded batch: the segments cover tokens [2, T - 3) with empty segments among them;
    the other tokens count as without an adapter."""
    d = dense_inputs(T, 136, 264, 4, 16, dt, "silu", True, True, 3)
    mid = T // 2
    d["offs"] = torch.tensor([2, 2, mid, mid, mid, T - 3, T - 3], dtype=torch.int32)
    d["segs"] = torch.tensor([3, 1, 0, 2, 2, 0], dtype=torch.int32)
    check_dense(d, run_dense(d))


@pytest.mark.parametrize("T", [12, 300])
def test_a_broken_adapter_stays_with_its_tenant(T):
    """Infinities and NaN in one tenant's A and B, and in one token's x: other tenants' tokens
    are what they were; the tenant's own follow the formula (not finite where it is not)."""
    for act in ("none", "silu_and_mul"):
        d = dense_inputs(T, 264, 328, 5, 16, BF16, act, True, True, 11, none_frac=0.1)
        rows = fr.row_adapters(T, d["offs"].numpy(), d["segs"].numpy())
        clean, _ = fr.dense_fused(*(d[k].double().numpy() for k in ("x", "w", "a", "b")), rows,
                                  bias=d["bias"].double().numpy(), act=act, residual=d["residual"].double().numpy(),
                                  lora_scale=d["scale"])
        d["b"][2, 3, 17], d["b"][2, 9, 250] = float("inf"), float("nan")
        d["b"][4, 15, 40] = float("-inf")
        d["a"][3, 5, 100] = float("nan")
        y = run_dense(d).float().cpu().numpy()
        other = (rows != 2) & (rows != 3) & (rows != 4)
        assert other.any() and np.isfinite(y[other]).all()
        good = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
        good["b"] = torch.nan_to_num(d["b"], 0.0, 0.0, 0.0)
        good["a"] = torch.nan_to_num(d["a"], 0.0)
        check_dense(good, torch.from_numpy(y), where=np.flatnonzero(other))
        h_out = y.shape[1]
        touched = np.zeros(h_out, bool)
        for f in (17, 250):
            touched[f % h_out if act == "silu_and_mul" else f] = True
        assert np.isnan(y[rows == 3]).all()
        assert not np.isfinite(y[rows == 2][:, 250 % h_out]).any()
        rest = np.ix_(np.flatnonzero(rows == 2), np.flatnonzero(~touched))
        check_dense(good, torch.from_numpy(y), where=rest)


@pytest.mark.parametrize("row", [3, 64, 127])
@pytest.mark.parametrize("T,K", [(12, 520), (40, 520), (150, 520), (300, 520), (300, 264), (900, 264)])
def test_a_broken_half_of_a_wide_adapter(T, K, row):
    """Rank 128, one infinity in either half of the rank rows: the tenant's features beside it
    still get every rank row once."""
    d = dense_inputs(T, K, 328, 5, 128, BF16, "none", True, True, 11, none_frac=0.1)
    good = dict(d, b=d["b"].clone())
    rows = fr.row_adapters(T, d["offs"].numpy(), d["segs"].numpy())
    assert (rows == 2).any()
    d["b"][2, row, 17], good["b"][2, row, 17] = float("inf"), 0.0
    y = run_dense(d).float().cpu()
    assert not torch.isfinite(y[torch.from_numpy(rows == 2), 17]).any()
    check_dense(good, y, where=np.ix_(np.arange(T), np.flatnonzero(np.arange(328) != 17)))
    check_dense(good, y, where=np.flatnonzero(rows != 2))


@pytest.mark.parametrize("T", [5, 300])
def test_a_token_that_is_not_finite_stays_alone(T):
    d = dense_inputs(T, 264, 328, 3, 16, BF16, "gelu", True, True, 2)
    want = run_dense(d)
    d["x"][2, 100] = float("nan")
    d["x"][4, 7] = float("inf")
    got = run_dense(d)
    keep = [t for t in range(T) if t not in (2, 4)]
    assert torch.equal(want[keep], got[keep]) and torch.isnan(got[2]).all()


@pytest.mark.parametrize("T", [9, 64, 300, 1100])
def test_in_place_residual(T):
    """y is the residual: the same values as with a y of its own."""
    for act in ("none", "silu_and_mul"):
        d = dense_inputs(T, 264, 520, 3, 16, BF16, act, True, True, T)
        want = run_dense(d)
        q = {k: dev(v) for k, v in d.items()}
        y = q["residual"].clone()
        got = ml.dense_lora_fused(q["x"], q["w"], q["a"], q["b"], q["offs"], q["segs"], bias=q["bias"],
                                  activation=act, residual=y, lora_scale=d["scale"], y=y)
        assert got.data_ptr() == y.data_ptr() and torch.equal(want, got)


@pytest.mark.parametrize("T", [1, 64, 300])
def test_same_bits_twice(T):
    d = dense_inputs(T, 1032, 520, 4, 32, BF16, "gelu_tanh", True, True, T)
    a, b = run_dense(d), run_dense(d)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T", [20, 300])
def test_bad_segments_are_flagged(T, dt):
    d = dense_inputs(T, 72, 136, 3, 8, dt, "none", False, False, 1)
    d["offs"] = torch.tensor([0, 4, 8, T], dtype=torch.int32)
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, T, 72, 136, 1, 1, 3, 8), "cuda")
    for segs, offs in ([1, 7, 2], [0, 4, 8, T]), ([1, 0, 2], [0, 8, 4, T]), ([1, 0, -3], [0, 4, 8, T]), \
            ([1, 0, 2], [0, 4, 8, T + 5]), ([1, 0, 2], [-2, 4, 8, T]):
        d["segs"], d["offs"] = torch.tensor(segs, dtype=torch.int32), torch.tensor(offs, dtype=torch.int32)
        y = run_dense(d, workspace=ws)
        with pytest.raises(ml.MoELoRAError) as ei:
            ml.check_status(ws)
        assert ei.value.status == ml.ERR_DEVICE_CHECK
        assert torch.isfinite(y).all()
    # the next good call on the workspace is clean
    d["segs"], d["offs"] = torch.tensor([1, 0, 2], dtype=torch.int32), torch.tensor([0, 4, 8, T], dtype=torch.int32)
    check_dense(d, run_dense(d, workspace=ws))
    ml.check_status(ws)


def test_no_tokens():
    d = dense_inputs(1, 72, 136, 0, 0, BF16, "none", False, False, 1)
    y = ml.dense_lora_fused(d["x"][:0].cuda(), d["w"].cuda())
    assert y.shape == (0, 136)


def test_buffers_of_the_caller():
    """Rows of y behind T and bytes behind the workspace stay as they were."""
    for T in (5, 300):
        for dt in (BF16, F32):
            d = dense_inputs(T, 136, 264, 3, 16, dt, "silu_and_mul", True, True, 1)
            need = ml.workspace_size(ml.OP_DENSE_FUSED, T, 136, 264, 1, 1, 3, 16)
            ws = torch.full((need + 256,), 171, dtype=torch.uint8, device="cuda")
            big = torch.full((T + 3, 264), 77.0, dtype=dt, device="cuda")
            y = run_dense(d, workspace=ws[:need], y=big[:T])
            check_dense(d, y)
            assert (big[T:] == 77.0).all() and (ws[need:] == 171).all()


@pytest.mark.parametrize("T", [8, 300])
def test_captured_and_replayed(T):
    """Two graphs on one workspace, replayed in turn with new inputs and new segments."""
    d = dense_inputs(T, 264, 392, 4, 16, BF16, "silu", True, True, 1, grouped=False)
    S = d["segs"].numel()
    e = dense_inputs(T, 264, 392, 4, 16, BF16, "gelu", True, True, 1, grouped=False)
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, T, 264, 392, 1, 1, 4, 16), "cuda")
    q = {k: dev(v) for k, v in d.items()}
    call = lambda act: ml.dense_lora_fused(q["x"], q["w"], q["a"], q["b"], q["offs"], q["segs"], bias=q["bias"],
                                           activation=act, residual=q["residual"], lora_scale=0.5, workspace=ws)
    call("silu")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for act in ("silu", "gelu"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(act))
        graphs.append(g)
    for seed in (5, 6):
        n = dense_inputs(T, 264, 392, 4, 16, BF16, "silu", True, True, seed)
        perm = np.random.default_rng(seed).permutation(S)
        d["x"], d["segs"] = n["x"], d["segs"][torch.from_numpy(perm)]
        q["x"].copy_(d["x"])
        q["segs"].copy_(d["segs"])
        for g, o, act in zip(graphs, outs, ("silu", "gelu")):
            g.replay()
            torch.cuda.synchronize()
            check_dense({**d, "act": act}, o)


def test_two_streams_at_once():
    """Two calls with workspaces of their own, on two streams at the same time."""
    ds = [dense_inputs(T, 520, 776, 4, 16, BF16, act, True, True, T) for T, act in ((48, "silu"), (700, "silu_and_mul"))]
    qs = [{k: dev(v) for k, v in d.items()} for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(5):
        for i, (d, q, s) in enumerate(zip(ds, qs, streams)):
            outs[i] = ml.dense_lora_fused(q["x"], q["w"], q["a"], q["b"], q["offs"], q["segs"], bias=q["bias"],
                                          activation=d["act"], residual=q["residual"], lora_scale=0.5, stream=s)
    torch.cuda.synchronize()
    for d, o in zip(ds, outs):
        check_dense(d, o)


def test_operators_together():
    """A block as it is served: scored routing, the routed experts, then the shared expert that
    every token passes, its down projection adding to the experts' output in place."""
    from tests.gpu_cases import moe_weights_both
    from workloads import synth
    s = synth.MoEShape("block", 401, E=16, k=4, H=256, I=192, L=3, r=16, no_adapter_frac=0.25)
    for M in (1, 30, 400):
        cpu, w, OW = moe_weights_both(s)
        x, wr, lg = grid_router(M, s.E, s.H, M)
        ids_ad = np.sort(adapters(M, s.L, M))
        ad = torch.from_numpy(ids_ad)
        sb = np.random.default_rng(M).standard_normal(s.E).astype(np.float32) * 0.1
        fmt = dict(score="sigmoid", n_group=4, topk_group=2, group_rule="top2", scale=2.5)
        rt = ml.route_scored(ad.cuda(), s.k, s.L, x=x.cuda(), w_router=wr.cuda(),
                             score_bias=torch.from_numpy(sb).cuda(), **fmt)
        check_route(rt, lg, ids_ad, s.E, s.k, s.L, score_bias=sb.astype(np.float64), **fmt)
        y = ml.forward(x.cuda(), rt, w, k=s.k, L=s.L)
        gu = dense_inputs(M, s.H, 320, s.L, 16, BF16, "silu_and_mul", False, False, 3)
        dn = dense_inputs(M, 320, s.H, s.L, 16, BF16, "none", True, False, 4)
        st = [0] + [i for i in range(1, M) if ids_ad[i] != ids_ad[i - 1]]
        offs, segs = torch.tensor(st + [M], dtype=torch.int32), torch.from_numpy(ids_ad[st].astype(np.int32))
        seg = (offs.cuda(), segs.cuda())
        act = ml.dense_lora_fused(x.cuda(), gu["w"].cuda(), gu["a"].cuda(), gu["b"].cuda(), *seg,
                                  activation="silu_and_mul", lora_scale=0.5)
        out = ml.dense_lora_fused(act, dn["w"].cuda(), dn["a"].cuda(), dn["b"].cuda(), *seg, bias=dn["bias"].cuda(),
                                  residual=y, lora_scale=0.5, y=y)
        torch.cuda.synchronize()
        f = lambda t: t.double().numpy()
        ids, wts = fr.route_scored(lg, s.k, score_bias=sb.astype(np.float64), **fmt)
        routed = ref.moe_lora_forward(f(x), ids, wts, ids_ad.astype(np.int64), s.I, OW.expert, OW.adapter,
                                      tokens=np.arange(M))
        a64, _ = fr.dense_fused(f(x), f(gu["w"]), f(gu["a"]), f(gu["b"]), ids_ad, act="silu_and_mul", lora_scale=0.5)
        want, _ = fr.dense_fused(a64, f(dn["w"]), f(dn["a"]), f(dn["b"]), ids_ad, bias=f(dn["bias"]),
                                 residual=routed, lora_scale=0.5)
        assert rel_err(out, want) <= TOL_BF16


@pytest.mark.parametrize("T,h_in,h_out", [(468, 1576, 864), (130, 2048, 200), (7, 1032, 2048), (512, 264, 1000)])
def test_larger_sizes_f32(T, h_in, h_out):
    """Every split of h_in, tiles that end inside a block."""
    _check(T, h_in, h_out, 3, 8, F32, "gelu", True, True, T)
    _check(T, h_in, h_out, 2, 128, F32, "silu_and_mul", True, False, T)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T", [1, 64, 200, 300, 1100])
def test_calls_that_feed_each_other(T, dt):
    """A chain without a pause, each call reading what the one before wrote, a torch kernel among
    them: the same bits as with a synchronisation after every call."""
    ds = [dense_inputs(T, 520, 520, 4, r, dt, act, True, True, i, grouped=g)
          for i, (r, act, g) in enumerate([(16, "gelu", True), (64, "silu", False), (8, "relu", True)])]
    bare = dense_inputs(T, 520, 520, 0, 0, dt, "none", True, True, 9)
    qs = [{k: dev(v) for k, v in d.items()} for d in ds + [bare]]
    ws = ml.new_workspace(max(ml.workspace_size(ml.OP_DENSE_FUSED, T, 520, 520, 1, 1, 4, r) for r in (8, 16, 64)), "cuda")

    def chain(pause):
        h = qs[0]["x"]
        for _ in range(6):
            for q, act in zip(qs, ("gelu", "silu", "relu", "none")):
                h = ml.dense_lora_fused(h, q["w"], q["a"], q["b"], q["offs"], q["segs"], bias=q["bias"],
                                        activation=act, residual=q["residual"], lora_scale=0.5, workspace=ws)
                pause()
            h = h / 2
            pause()
        return h

    want = chain(torch.cuda.synchronize)
    torch.cuda.synchronize()
    for _ in range(4):
        got = chain(lambda: None)
        assert torch.equal(got, want)


def test_offsets_past_32_bits():
    """An output of more than 2^31 elements: its last rows are what they are on their own."""
    T, K, N = 270001, 64, 8192
    d = dense_inputs(64, K, N, 2, 8, BF16, "silu", True, False, 5, grouped=False)
    rows = fr.row_adapters(64, d["offs"].numpy(), d["segs"].numpy())
    x = torch.zeros((T, K), dtype=BF16, device="cuda")
    x[-64:] = d["x"].cuda()
    offs = torch.cat([torch.zeros(1, dtype=torch.int32), d["offs"] + (T - 64)])
    segs = torch.cat([torch.full((1,), -1, dtype=torch.int32), d["segs"]])
    y = ml.dense_lora_fused(x, d["w"].cuda(), d["a"].cuda(), d["b"].cuda(), offs.cuda(), segs.cuda(),
                            bias=d["bias"].cuda(), activation="silu", lora_scale=d["scale"])
    assert y.numel() > 2 ** 31
    check_dense(d, y[-64:], rows)
    assert torch.equal(y[0], y[1000]) and torch.equal(y[0], y[T - 65])  # rows of zeros: act(bias)


def test_captured_on_two_branches():
    """One graph whose branches run side by side and join: calls first on a branch, behind a copy,
    behind a torch kernel, and behind two branches at once."""
    T = 70
    a = dense_inputs(T, 264, 392, 3, 16, BF16, "silu", True, True, 1)
    b = dense_inputs(300, 264, 392, 3, 16, BF16, "gelu", True, False, 2)
    c = dense_inputs(T, 392, 264, 0, 0, BF16, "none", True, False, 3)
    f = dense_inputs(T, 264, 136, 2, 8, F32, "none", True, False, 4)
    qs = [{k: dev(v) for k, v in d.items()} for d in (a, b, c, f)]
    lg = torch.from_numpy(np.random.default_rng(1).standard_normal((200, 16)).astype(np.float32)).cuda()
    ad = torch.from_numpy(adapters(200, 3, 1)).cuda()

    def call(q, x=None):
        return ml.dense_lora_fused(q["x"] if x is None else x, q["w"], q["a"], q["b"], q["offs"], q["segs"],
                                   bias=q["bias"], activation=q["act"], residual=q["residual"], lora_scale=0.5)

    def work(main, side):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            xb = qs[1]["x"].clone()
            y1 = call(qs[1], xb)
            r = ml.route_scored(ad, 3, 3, logits_in=lg, score="sigmoid")
            y3 = call(qs[3])
        y0 = call(qs[0])
        h = y0 + 0
        main.wait_stream(side)
        y2 = call(qs[2], h)
        return y0, y1, y2, y3, r["topk_ids"], r["sorted_pairs"]

    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        want = work(main, side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        got = work(main, side)
    for _ in range(3):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
    for d, o in ((a, got[0]), (b, got[1]), (f, got[3])):
        check_dense(d, o)


@pytest.mark.parametrize("act", ["gelu", "silu_and_mul"])
@pytest.mark.parametrize("T,h_in,h_out", [(257, 1032, 72), (300, 2048, 1024), (513, 4104, 136), (1000, 520, 520),
                                          (2100, 2056, 200)])
def test_more_tokens_with_few_tiles(T, h_in, h_out, act):
    """Several blocks of 256 tokens whose reduction is split, adapters in each."""
    _check(T, h_in, h_out, 5, 16, BF16, act, True, True, T)
    _check(T, h_in, h_out, 3, 128, BF16, act, False, False, T + 1)
    _check(T, h_in, h_out, 0, 0, BF16, act, True, False, T + 2)
    d = dense_inputs(T, h_in, h_out, 20, 8, BF16, act, False, True, T, grouped=False)
    check_dense(d, run_dense(d))


def test_a_broken_adapter_among_few_tiles():
    T = 700
    d = dense_inputs(T, 2056, 136, 5, 16, BF16, "none", True, True, 3, none_frac=0.1)
    rows = fr.row_adapters(T, d["offs"].numpy(), d["segs"].numpy())
    good = dict(d, b=d["b"].clone())
    d["b"][2, 3, 17], good["b"][2, 3, 17] = float("inf"), 0.0
    y = run_dense(d).float().cpu()
    assert not torch.isfinite(y[torch.from_numpy(rows == 2), 17]).any()
    check_dense(good, y, where=np.ix_(np.arange(T), np.flatnonzero(np.arange(136) != 17)))
    check_dense(good, y, where=np.flatnonzero(rows != 2))


@pytest.mark.parametrize("act", ["silu", "silu_and_mul"])
@pytest.mark.parametrize("T,r", [(1, 8), (1, 16), (2, 8), (1, 32), (1, 128), (2, 16), (3, 8), (4, 16)])
@pytest.mark.parametrize("h_in,h_out", [(8, 8), (72, 200), (4104, 1000), (11008, 264)])
def test_a_token_or_a_few(T, r, h_in, h_out, act):
    """The smallest calls, over every split of the reduction."""
    _check(T, h_in, h_out, 6, r, BF16, act, True, True, T + r, none_frac=0.0, grouped=False)
    _check(T, h_in, h_out, 6, r, BF16, act, False, False, T + r + 1, none_frac=0.5, grouped=False)


@pytest.mark.parametrize("r", [8, 16, 128])
def test_one_tokens_broken_adapter_and_segments(r):
    d = dense_inputs(2, 520, 264, 4, r, BF16, "none", True, False, 1)
    d["offs"], d["segs"] = torch.tensor([0, 1, 2], dtype=torch.int32), torch.tensor([2, 1], dtype=torch.int32)
    good = dict(d, b=d["b"].clone())
    d["b"][2, 5, 40], good["b"][2, 5, 40] = float("nan"), 0.0
    y = run_dense(d).float().cpu()
    assert torch.isnan(y[0, 40])
    check_dense(good, y, where=np.ix_([0], np.flatnonzero(np.arange(264) != 40)))
    check_dense(good, y, where=[1])
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, 2, 520, 264, 1, 1, 4, r), "cuda")
    for segs, offs in ([2, 9], [0, 1, 2]), ([2, 1], [0, 2, 1]), ([2, 1], [0, 1, 7]):
        bad = dict(good, segs=torch.tensor(segs, dtype=torch.int32), offs=torch.tensor(offs, dtype=torch.int32))
        assert torch.isfinite(run_dense(bad, workspace=ws)).all()
        with pytest.raises(ml.MoELoRAError) as ei:
            ml.check_status(ws)
        assert ei.value.status == ml.ERR_DEVICE_CHECK
    check_dense(good, run_dense(good, workspace=ws))
    ml.check_status(ws)
