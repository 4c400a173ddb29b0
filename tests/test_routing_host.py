"""Routing objects on the host: the fields are all tensors, and the mark of an expert
share goes along with copies."""
from dataclasses import fields

import pytest
import torch

import routing_grouped_expert_amd as moe


def test_fields_are_the_eight_tensors():
    r = moe.Routing.empty(6, 4, 2, torch.float32, "cpu")
    assert r.layer_experts is None
    copy = moe.Routing(**{k: v.clone() for k, v in vars(r).items()})
    assert [f.name for f in fields(copy)] == list(vars(copy))
    assert all(a is b for a, b in zip(r.tensors(), (getattr(r, f.name) for f in fields(r))))
    assert len(r.tensors()) == 8 and copy.layer_experts is None


def test_the_mark_of_a_share_goes_along():
    r = moe.Routing.empty(6, 4, 2, torch.float32, "cpu")
    r.layer_experts = 16
    copy = moe.Routing(**vars(r))
    assert copy.layer_experts == 16
    assert moe.Routing.empty(6, 4, 2, torch.float32, "cpu").layer_experts is None
    x = torch.zeros(6, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="share"):
        moe.moe_experts_int4(x, x, x, None, x, x, None, copy, "silu")
