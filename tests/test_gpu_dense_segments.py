"""Segments of dense_lora_fused that are wrong in every way at once: flagged, and every token
counts by the last segment that begins at or before it, if it ends behind it."""
import bisect

import numpy as np
import pytest
import torch

import moe_lora_b200 as ml
from oracle import fused_ref as fr
from tests.fused_cases import run_dense
from tests.grid_cases import check_grid, grid_inputs

pytestmark = pytest.mark.gpu


def _overlapping(S, T, L, none):
    """Offsets that swing between 0 and T: each second segment holds every token."""
    offs = np.where(np.arange(S + 1) % 2 == 0, 0, T).astype(np.int32)
    segs = (np.arange(S) % (L + none)).astype(np.int32)
    segs[segs >= L] = -1
    return offs, segs


def _rows(offs, segs, T):
    """What the kernels' binary search finds for each token."""
    rows = np.full(T, -1, dtype=np.int64)
    for t in range(T):
        lo, hi = 0, len(segs)
        while hi - lo > 1:
            mid = (lo + hi) // 2
            lo, hi = (mid, hi) if offs[mid] <= t else (lo, mid)
        if offs[lo] <= t < offs[lo + 1]:
            rows[t] = segs[lo]
    return rows


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [5, 64, 200, 300])
@pytest.mark.parametrize("S", [3, 700, 60000])
def test_segments_that_overlap(S, T, dt):
    d = grid_inputs(T, 264, 136, 5, 16, dt, "none", True, True, T)
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, T, 264, 136, 1, 1, 5, 16), "cuda")
    for none in (0, 1):
        offs, segs = _overlapping(S, T, 5, none)
        bad = dict(d, offs=torch.from_numpy(offs), segs=torch.from_numpy(segs))
        check_grid(bad, run_dense(bad, workspace=ws), _rows(offs, segs, T))
        with pytest.raises(ml.MoELoRAError) as ei:
            ml.check_status(ws)
        assert ei.value.status == ml.ERR_DEVICE_CHECK


@pytest.mark.parametrize("T", [5, 64, 300])
def test_many_empty_segments(T):
    """As many segments as tokens a hundred times over, most of them empty."""
    g = np.random.default_rng(T)
    S = 100 * T
    offs = np.concatenate([[0], np.sort(g.integers(0, T + 1, S - 1)), [T]]).astype(np.int32)
    segs = g.integers(-1, 5, S).astype(np.int32)
    d = grid_inputs(T, 264, 136, 5, 16, torch.bfloat16, "none", True, True, T)
    d["offs"], d["segs"] = torch.from_numpy(offs), torch.from_numpy(segs)
    rows = np.array([segs[bisect.bisect_right(offs.tolist(), t) - 1] for t in range(T)])
    assert np.array_equal(rows, fr.row_adapters(T, offs, segs))
    ws = ml.new_workspace(ml.workspace_size(ml.OP_DENSE_FUSED, T, 264, 136, 1, 1, 5, 16), "cuda")
    check_grid(d, run_dense(d, workspace=ws), rows)
    ml.check_status(ws)
