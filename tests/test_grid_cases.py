"""What the tolerances of the exact inputs can see: a lost piece of a sum, one rounding too many."""
import numpy as np
import pytest
import torch

from oracle import fused_ref as fr
from tests.fused_cases import dense_oracle
from tests.grid_cases import EDGES, FEW, SIZES, grid_inputs, grid_tolerance


class Case:
    """A projection whose h can be spoilt: the error of the output in units of its tolerance."""

    def __init__(self, T, h_in, h_out, L, r, dt, act):
        self.d = d = grid_inputs(T, h_in, h_out, L, r, dt, act, True, True, T + h_in, none_frac=0.0)
        self.y, self.m = dense_oracle(d)
        self.tol = grid_tolerance(d, self.y, self.m)
        self.rows = fr.row_adapters(T, d["offs"].numpy(), d["segs"].numpy())
        self.f = {k: d[k].double().numpy() for k in ("x", "w", "a", "b", "residual")}
        self.used = sorted(set(self.rows.tolist()))

    def z(self, ad):
        t = np.flatnonzero(self.rows == ad)
        return t, self.d["scale"] * (self.f["x"][t] @ self.f["a"][ad].T)

    def error(self, missing):
        y = fr.activation(self.d["act"], self.m["h"] - missing, self.y.shape[1]) + self.f["residual"]
        y = torch.from_numpy(y).float().to(self.d["x"].dtype).double().numpy()
        return float(np.max(np.abs(y - self.y) / self.tol))

    def columns(self, k0, k1):  # columns of x and W
        return self.f["x"][:, k0:k1] @ self.f["w"][:, k0:k1].T

    def ranks(self, adapters, i0=0, i1=None):  # rank rows of adapters
        out = np.zeros_like(self.m["h"])
        for ad in adapters:
            t, z = self.z(ad)
            out[t] = z[:, i0:i1] @ self.f["b"][ad][i0:i1]
        return out


@pytest.mark.parametrize("T,h_in,h_out,L,r,act", [(*s, a) for s in SIZES for a in ("none", "silu_and_mul")] +
                         [(*s, "none") for s in FEW + EDGES])
def test_lost_pieces_are_seen(T, h_in, h_out, L, r, act):
    c = Case(T, h_in, h_out, L, r, torch.bfloat16, act)
    assert c.error(0.0) <= 1.0
    nkb = (h_in + 63) // 64
    for kb in {0, nkb // 2, nkb - 1}:  # a K block
        assert c.error(c.columns(64 * kb, 64 * kb + 64)) > 1.5
    for ad in {c.used[0], c.used[-1]}:  # a step of 16 ranks
        for i in range(0, r, 16):
            assert c.error(c.ranks([ad], i, i + 16)) > 1.5
    per = max(1, 32 // r)  # a group of adapters, lost or taken twice
    for first in range(0, len(c.used), per):
        part = c.ranks(c.used[first:first + per])
        assert c.error(part) > 1.5 and c.error(-part) > 1.5


# (one token has too few outputs for one of them to lie that close to a border)
@pytest.mark.parametrize("T,h_in,h_out,L,r", [s for s in SIZES if s[0] > 1])
def test_z_of_eight_bits_is_seen(T, h_in, h_out, L, r):
    c = Case(T, h_in, h_out, L, r, torch.bfloat16, "none")
    off = np.zeros_like(c.m["h"])
    for ad in c.used:
        t, z = c.z(ad)
        off[t] = (z - torch.from_numpy(z).float().to(torch.bfloat16).double().numpy()) @ c.f["b"][ad]
    assert c.error(off) > 1.0


@pytest.mark.parametrize("T,h_in,h_out,L,r", [(19, 2048, 136, 4, 8), (512, 2048, 264, 2, 64)])
def test_pieces_lost_in_fp32_are_seen(T, h_in, h_out, L, r):
    c = Case(T, h_in, h_out, L, r, torch.float32, "silu_and_mul")
    assert c.error(0.0) <= 1.0
    assert c.error(c.columns(h_in - 8, h_in)) > 100
    assert c.error(c.ranks([c.used[0]], r - 1, r)) > 100
