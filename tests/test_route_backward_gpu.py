"""The softmax gradient where a routing of the caller's own names an expert in several
slots of a token: the logit has the sum of the slots' gradients.

A slot's gradient is off by at most (k + 4) 2^-24 of its terms' magnitudes (as in
test_sorted_rows_gpu.py), the sum of up to k slots by k more, then one rounding."""
import numpy as np
import pytest
import torch

from routing_grouped_expert_amd import Routing, moe_route_backward

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,e,k", [(1, 4, 2), (50, 3, 3), (33, 8, 8), (70, 37, 16)])
def test_slots_of_one_expert_add_up(n, e, k, dt):
    print(f"[route-grad] n={n} E={e} k={k} {dt}", flush=True)
    g = torch.Generator().manual_seed(n * k)
    idx = torch.randint(0, min(e, max(2, k // 2)), (n, k), generator=g)
    w = torch.softmax(torch.randn(n, k, generator=g), 1).to(dt)
    dw = torch.randn(n, k, generator=g)
    r = Routing.empty(n, e, k, dt, DEV)
    r.topk_idx.copy_(idx)
    r.topk_w.copy_(w)
    got = moe_route_backward(dw.to(DEV), r).double().cpu().numpy()
    wd, dwd = w.double().numpy(), dw.double().numpy()
    slot = wd * (dwd - (wd * dwd).sum(1, keepdims=True))
    mag = wd * (np.abs(dwd) + (wd * np.abs(dwd)).sum(1, keepdims=True))
    want, terms = np.zeros((n, e)), np.zeros((n, e))
    for t in range(n):
        np.add.at(want[t], idx[t].numpy(), slot[t])
        np.add.at(terms[t], idx[t].numpy(), mag[t])
    tol = torch.finfo(dt).eps / 2 * (1 + 1e-3) * np.abs(want) + (2 * k + 4) * 2.0 ** -24 * terms
    assert (np.abs(got - want) <= tol).all()
