"""GPU parity of moe_lora_route_scored against the fp64 oracle: ids, pairs and offsets exact,
weights within fp32 rounding."""
import numpy as np
import pytest
import torch

import moe_lora_b200 as ml
from oracle import fused_ref as fr
from tests.fused_cases import adapters, check_route, grid_router

pytestmark = pytest.mark.gpu


def _run(lg, ad, k, L, score_bias=None, **fmt):
    sb = None if score_bias is None else torch.from_numpy(np.asarray(score_bias, dtype=np.float32)).cuda()
    res = ml.route_scored(torch.from_numpy(ad).cuda(), k, L, logits_in=torch.from_numpy(lg).cuda(),
                          score_bias=sb, want_logits=True, **fmt)
    torch.cuda.synchronize()
    return res


def _check(M, E, k, L, seed, lg=None, score_bias=None, status=True, **fmt):
    g = np.random.default_rng(seed)
    if lg is None:
        lg = g.standard_normal((M, E)).astype(np.float32)
    ad = adapters(M, L, seed + 1)
    res = _run(lg, ad, k, L, score_bias, **fmt)
    check_route(res, lg.astype(np.float64), ad, E, k, L,
                score_bias=None if score_bias is None else np.asarray(score_bias, np.float32).astype(np.float64),
                **fmt)
    assert np.array_equal(res["logits"].cpu().numpy(), lg, equal_nan=True)
    if status:
        ml.check_status(res["workspace"])
    return res


SHAPES = [(1, 64, 8, 8), (1, 1, 1, 0), (2, 5, 5, 1), (7, 8, 2, 64), (37, 20, 3, 3), (64, 128, 8, 32),
          (128, 256, 8, 64), (129, 96, 7, 5), (203, 256, 1, 16), (1000, 160, 6, 5), (4096, 128, 8, 16),
          (300, 64, 64, 2), (40, 256, 256, 4)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k,L", SHAPES)
def test_no_groups(M, E, k, L, score):
    _check(M, E, k, L, M + E, score=score, renormalize=True, scale=1.0)
    b = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.1
    _check(M, E, k, L, M + E + 1, score=score, score_bias=b, renormalize=False, scale=2.5)


@pytest.mark.parametrize("rule", ["max", "top2"])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("M,E,k,L,n_group,topk_group", [
    (1, 64, 8, 8, 8, 4), (64, 128, 8, 32, 8, 4), (33, 256, 8, 4, 8, 3), (777, 160, 6, 5, 10, 3),
    (50, 20, 2, 0, 20, 3),     # groups of one expert
    (50, 40, 5, 1, 8, 1),      # every expert of the one kept group
    (130, 256, 3, 2, 128, 60),  # more groups than lanes
    (70, 200, 10, 9, 4, 4)])   # every group kept
def test_groups(M, E, k, L, n_group, topk_group, score, biased, rule):
    b = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.05 if biased else None
    _check(M, E, k, L, M * 3 + E, score=score, score_bias=b, n_group=n_group, topk_group=topk_group,
           group_rule=rule, renormalize=biased, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_index(score, biased):
    g = np.random.default_rng(8)
    lg = (g.integers(-4, 5, size=(300, 32)) * 0.25).astype(np.float32)
    b = (g.integers(-1, 2, size=32) * 0.125).astype(np.float32) if biased else None
    _check(300, 32, 6, 4, 1, lg=lg, score=score, score_bias=b)
    _check(300, 32, 6, 4, 2, lg=lg, score=score, score_bias=b, n_group=8, topk_group=4, group_rule="top2")
    _check(50, 32, 6, 4, 3, lg=np.zeros((50, 32), np.float32), score=score, score_bias=b, n_group=4, topk_group=2)


def test_scores_closer_than_a_rounding():
    """Selection scores that differ by less than fp32 holds: the bias of expert e is moved by
    one float so that score + bias falls on either side of its neighbour's."""
    E, M = 64, 512
    g = np.random.default_rng(12)
    lg = g.standard_normal((M, E)).astype(np.float32)
    s0 = 1 / (1 + np.exp(-lg[0].astype(np.float64)))
    b = (0.9 - s0).astype(np.float32)  # row 0: every selection score within a rounding of 0.9
    _check(M, E, 8, 3, 4, lg=lg, score="sigmoid", score_bias=b)
    _check(M, E, 8, 3, 4, lg=lg, score="sigmoid", score_bias=b, n_group=8, topk_group=3, group_rule="top2")
    p = np.exp(lg[0].astype(np.float64))
    b = (0.5 - p / p.sum()).astype(np.float32)
    _check(M, E, 8, 3, 4, lg=lg, score="softmax", score_bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score):
    """-inf logits, rows with fewer experts than k, rows with none; +inf; saturated scores."""
    g = np.random.default_rng(9)
    lg = g.standard_normal((40, 24)).astype(np.float32)
    lg[g.random((40, 24)) < 0.7] = -np.inf
    lg[3] = -np.inf
    lg[4, 5:] = -np.inf
    lg[5] = np.finfo(np.float32).min
    lg[6, 2] = np.inf
    lg[7, [1, 9]] = np.inf
    lg[8] = -95 - np.arange(24)      # sigmoids below the smallest normal float
    lg[9] = 60 + np.arange(24)       # sigmoids that round to one
    for renorm in (True, False):
        _check(40, 24, 6, 2, 1, lg=lg, score=score, renormalize=renorm)
        _check(40, 24, 6, 2, 1, lg=lg, score=score, renormalize=renorm, n_group=4, topk_group=2, group_rule="max")
    b = np.zeros(24, np.float32)
    b[4], b[11] = -np.inf, np.inf
    _check(40, 24, 6, 2, 1, lg=lg, score=score, score_bias=b)
    _check(40, 24, 6, 2, 1, lg=lg, score=score, score_bias=b, n_group=6, topk_group=3, group_rule="top2")


@pytest.mark.parametrize("n_group", [1, 4])
def test_nan_is_the_last_choice_and_flagged(n_group):
    g = np.random.default_rng(10)
    lg = g.standard_normal((30, 16)).astype(np.float32)
    lg[2, 3] = np.nan
    lg[5, :14] = np.nan
    lg[6] = np.nan
    fmt = dict(score="sigmoid", n_group=n_group, topk_group=max(1, n_group // 2 + 1), group_rule="max")
    for b in (None, np.where(np.arange(16) == 7, np.nan, 0.1).astype(np.float32)):
        res = _check(30, 16, 4, 3, 1, lg=lg, score_bias=b, status=False, **fmt)
        with pytest.raises(ml.MoELoRAError) as ei:
            ml.check_status(res["workspace"])
        assert ei.value.status == ml.ERR_DEVICE_CHECK


def test_bad_adapter_id_is_flagged_and_counts_as_none():
    lg = np.random.default_rng(3).standard_normal((40, 8)).astype(np.float32)
    ad = np.zeros(40, np.int32)
    ad[3], ad[17] = 7, -5
    res = _run(lg, ad, 2, 2, score="sigmoid")
    with pytest.raises(ml.MoELoRAError) as ei:
        ml.check_status(res["workspace"])
    assert ei.value.status == ml.ERR_DEVICE_CHECK
    ok = np.where((ad < -1) | (ad >= 2), -1, ad)
    check_route(res, lg.astype(np.float64), ok, 8, 2, 2, score="sigmoid")


def test_no_tokens():
    res = ml.route_scored(torch.zeros(0, dtype=torch.int32, device="cuda"), 2, 3,
                          logits_in=torch.zeros((0, 8), device="cuda"), score="sigmoid")
    torch.cuda.synchronize()
    assert res["seg_offsets"].cpu().tolist() == [0] * 33 and res["sorted_pairs"].numel() == 0


FROM_X = [(1, 64, 8, 8, 2048), (1, 8, 2, 0, 8), (5, 20, 3, 2, 72), (64, 128, 8, 32, 7168), (100, 256, 8, 4, 520),
          (128, 256, 4, 64, 1032), (129, 64, 8, 8, 512), (255, 5, 5, 1, 264), (256, 128, 8, 16, 1024),
          (300, 200, 6, 3, 4096), (1000, 256, 8, 5, 136), (4096, 128, 8, 16, 4096), (5000, 256, 2, 2, 256)]


@pytest.mark.parametrize("M,E,k,L,H", FROM_X)
def test_from_x(M, E, k, L, H):
    """Logits computed by the call, exact by construction, so every id can be compared."""
    x, wr, lg = grid_router(M, E, H, M + E + H)
    ad = adapters(M, L, M)
    b = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.05
    n_group = 4 if E % 4 == 0 and k <= E // 2 else 1
    fmt = dict(score="sigmoid", n_group=n_group, topk_group=max(1, n_group // 2), group_rule="top2", scale=2.5)
    kw = dict(x=x.cuda(), w_router=wr.cuda(), score_bias=torch.from_numpy(b).cuda(), **fmt)
    res = ml.route_scored(torch.from_numpy(ad).cuda(), k, L, want_logits=True, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(res["logits"].cpu().numpy().astype(np.float64), lg)
    check_route(res, lg, ad, E, k, L, score_bias=b.astype(np.float64), **fmt)
    ml.check_status(res["workspace"])
    # without the logits, on the same workspace, the same bits
    again = ml.route_scored(torch.from_numpy(ad).cuda(), k, L, workspace=res["workspace"], **kw)
    for key in ("topk_ids", "topk_w", "sorted_pairs", "seg_offsets"):
        assert torch.equal(res[key], again[key])


@pytest.mark.parametrize("M", [3, 200])
def test_logit_bias(M):
    x, wr, lg = grid_router(M, 32, 256, 5)
    bias = (np.random.default_rng(6).integers(-16, 17, size=32) * 0.125).astype(np.float32)
    ad = adapters(M, 2, 1)
    res = ml.route_scored(torch.from_numpy(ad).cuda(), 4, 2, x=x.cuda(), w_router=wr.cuda(),
                          bias=torch.from_numpy(bias).cuda())
    torch.cuda.synchronize()
    check_route(res, lg + bias[None, :], ad, 32, 4, 2)


def test_defaults_agree_with_route():
    lg = torch.from_numpy(np.random.default_rng(4).standard_normal((500, 64)).astype(np.float32)).cuda()
    ad = torch.from_numpy(adapters(500, 4, 2)).cuda()
    a, b = ml.route(ad, 8, 4, logits_in=lg), ml.route_scored(ad, 8, 4, logits_in=lg)
    for key in ("topk_ids", "sorted_pairs", "seg_offsets"):
        assert torch.equal(a[key], b[key])
    torch.testing.assert_close(a["topk_w"], b["topk_w"], rtol=2.0 ** -16, atol=0)


@pytest.mark.parametrize("M", [16, 600])
def test_captured_and_replayed_on_another_stream(M):
    """Two graphs that share a workspace, replayed in turn on new inputs, on a side stream."""
    E, k, L, H = 64, 4, 3, 256
    x = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    xs, wr, _ = grid_router(M, E, H, 1)
    wr = wr.cuda()
    ad = torch.from_numpy(adapters(M, L, 1)).cuda()
    ws = ml.new_workspace(ml.workspace_size(ml.OP_ROUTE_SCORED, M, H, 0, E, k, L, 0), "cuda")
    side = torch.cuda.Stream()
    fmts = [dict(score="sigmoid"), dict(score="softmax", n_group=4, topk_group=2)]
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for f in fmts:
            ml.route_scored(ad, k, L, x=x, w_router=wr, workspace=ws, **f)  # first call outside the capture
        side.synchronize()
        for f in fmts:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(ml.route_scored(ad, k, L, x=x, w_router=wr, workspace=ws, **f))
            graphs.append(g)
        for seed in (2, 3):
            xs, _, _ = grid_router(M, E, H, seed)
            x.copy_(xs.cuda())
            lg = x.double().cpu().numpy() @ wr.double().cpu().numpy().T
            for g, o, f in zip(graphs, outs, fmts):
                g.replay()
                side.synchronize()
                check_route(o, lg, ad.cpu().numpy(), E, k, L, **f)


def test_buffers_of_the_caller():
    """out and workspace given; what lies behind them stays as it was."""
    M, E, k, L = 21, 16, 3, 2
    lg = np.random.default_rng(1).standard_normal((M, E)).astype(np.float32)
    ad = adapters(M, L, 1)
    big = {"topk_ids": torch.full((M + 4, k), -7, dtype=torch.int32, device="cuda"),
           "topk_w": torch.full((M + 4, k), -7.0, device="cuda"),
           "sorted_pairs": torch.full((M * k + 9,), -7, dtype=torch.int32, device="cuda"),
           "seg_offsets": torch.full((E * (L + 1) + 9,), -7, dtype=torch.int32, device="cuda")}
    need = ml.workspace_size(ml.OP_ROUTE_SCORED, M, 0, 0, E, k, L, 0)
    ws = torch.full((need + 256,), 171, dtype=torch.uint8, device="cuda")
    ml.route_scored(torch.from_numpy(ad).cuda(), k, L, logits_in=torch.from_numpy(lg).cuda(), score="sigmoid",
                    out=big, workspace=ws[:need])
    torch.cuda.synchronize()
    used = {"topk_ids": big["topk_ids"][:M], "topk_w": big["topk_w"][:M], "sorted_pairs": big["sorted_pairs"][:M * k],
            "seg_offsets": big["seg_offsets"][:E * (L + 1) + 1]}
    check_route(used, lg.astype(np.float64), ad, E, k, L, score="sigmoid")
    assert (big["topk_ids"][M:] == -7).all() and (big["topk_w"][M:] == -7).all()
    assert (big["sorted_pairs"][M * k:] == -7).all() and (big["seg_offsets"][E * (L + 1) + 1:] == -7).all()
    assert (ws[need:] == 171).all()


def test_every_token_on_one_expert():
    """A collapsed router: one expert holds every token, the largest batch of one key."""
    M, E, k, L = 9000, 64, 2, 1
    lg = np.random.default_rng(2).standard_normal((M, E)).astype(np.float32)
    lg[:, 17] = 9
    _check(M, E, k, L, 3, lg=lg, score="sigmoid")


@pytest.mark.parametrize("M", [1, 16, 127, 128, 129, 2049])
@pytest.mark.parametrize("E,L", [(3, 64), (33, 64), (256, 64), (256, 0)])
def test_every_adapter_and_expert_count(M, E, L):
    """Both sides of the one-launch limit, with as many adapters as there can be."""
    _check(M, E, min(E, 3), L, M + E + L, score="sigmoid",
           score_bias=np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.05)


def test_rows_of_nan_without_renormalisation():
    lg = np.random.default_rng(1).standard_normal((200, 12)).astype(np.float32)
    lg[7] = np.nan
    for M in (20, 200):
        for score in ("softmax", "sigmoid"):
            res = _check(M, 12, 3, 2, 1, lg=lg[:M], score=score, renormalize=False, status=False)
            with pytest.raises(ml.MoELoRAError):
                ml.check_status(res["workspace"])


@pytest.mark.parametrize("M", [40, 700])
def test_huge_biases_of_both_signs(M):
    """Group sums whose terms cancel, and experts a bias rules out or forces."""
    g = np.random.default_rng(5)
    lg = g.standard_normal((M, 32)).astype(np.float32)
    b = (g.standard_normal(32) * 0.05).astype(np.float32)
    b[[1, 9, 17]], b[[2, 10, 30]] = 3e6, -3e6
    for rule in ("max", "top2"):
        _check(M, 32, 5, 3, 2, lg=lg, score="sigmoid", score_bias=b, n_group=4, topk_group=3, group_rule=rule)
        _check(M, 32, 5, 3, 2, lg=lg, score="softmax", score_bias=b, n_group=8, topk_group=3, group_rule=rule)


@pytest.mark.parametrize("M,H", [(9473, 8), (9600, 72), (10001, 264), (12345, 128)])
@pytest.mark.parametrize("E", [20, 96, 256])
def test_pairs_of_tiles(M, H, E):
    """Batches whose tiles fill the SMs: two CTAs share 256 tokens."""
    x, wr, lg = grid_router(M, E, H, M + E)
    ad = adapters(M, 5, M)
    b = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.05
    bias = (np.random.default_rng(6).integers(-16, 17, size=E) * 0.125).astype(np.float32)
    fmt = dict(score="sigmoid", n_group=4, topk_group=2, group_rule="max", scale=2.5)
    res = ml.route_scored(torch.from_numpy(ad).cuda(), 4, 5, x=x.cuda(), w_router=wr.cuda(),
                          bias=torch.from_numpy(bias).cuda(), score_bias=torch.from_numpy(b).cuda(),
                          want_logits=True, **fmt)
    torch.cuda.synchronize()
    assert np.array_equal(res["logits"].cpu().numpy().astype(np.float64), lg + bias[None, :])
    check_route(res, lg + bias[None, :], ad, E, 4, 5, score_bias=b.astype(np.float64), **fmt)
    ml.check_status(res["workspace"])


@pytest.mark.parametrize("M", [9, 300, 9500])
def test_calls_that_follow_each_other(M):
    """Routing and sorting without a pause on one workspace and one set of outputs, the inputs
    rewritten between the calls."""
    E, k, L, H = 48, 4, 6, 256
    xs, wr, _ = grid_router(M, E, H, 3)
    xs, wr = xs.cuda(), wr.cuda()
    ads = [torch.from_numpy(adapters(M, L, s)).cuda() for s in range(3)]
    x, ad = torch.empty_like(xs), torch.empty_like(ads[0])
    ws = ml.new_workspace(ml.workspace_size(ml.OP_ROUTE_SCORED, M, H, 0, E, k, L, 0), "cuda")
    out = {key: torch.empty_like(v) for key, v in
           ml.route_scored(ads[0], k, L, x=xs, w_router=wr, score="sigmoid").items() if key != "workspace"}

    def run(pause):
        got = []
        for i in range(6):
            x.copy_(xs.roll(i, 0))
            ad.copy_(ads[i % 3])
            pause()
            o = ml.route_scored(ad, k, L, x=x, w_router=wr, score="sigmoid" if i % 2 else "softmax", n_group=4,
                                topk_group=2, out=out, workspace=ws)
            pause()
            got.append([o[key].clone() for key in ("topk_ids", "topk_w", "sorted_pairs", "seg_offsets")])
        return got

    want = run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    for a, b in zip(run(lambda: None), want):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M", [60, 1500])
def test_logits_of_few_bits(M, score):
    """Logits rounded to bf16, as many routers give them: ties among the first k and at the
    borders of groups in most rows."""
    lg = torch.from_numpy(np.random.default_rng(M).standard_normal((M, 64)).astype(np.float32) * 3)
    lg = lg.to(torch.bfloat16).float().numpy()
    _check(M, 64, 8, 3, 1, lg=lg, score=score)
    _check(M, 64, 8, 3, 2, lg=lg, score=score, n_group=8, topk_group=4, group_rule="max")
    _check(M, 64, 8, 3, 3, lg=lg, score=score, n_group=8, topk_group=4, group_rule="top2", renormalize=False)
