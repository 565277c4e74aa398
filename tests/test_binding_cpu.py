"""The bindings of scored routing and the fused projection, as far as they go without a GPU."""
import torch

from moe_lora_b200 import _lib


def test_a_changed_scale_is_seen():
    """A scale held in a tensor is read on every call, not once per tensor."""
    scale, groups = torch.tensor(2.5), torch.tensor(4)
    at = lambda: _lib._route_format("sigmoid", groups, 2, "top2", True, scale)
    assert (at().scale, at().n_group) == (2.5, 4)
    scale.mul_(2)
    groups.mul_(2)
    assert (at().scale, at().n_group) == (5.0, 8)
    assert at() is at()  # equal arguments share one format
