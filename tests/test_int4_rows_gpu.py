"""4-bit experts with uneven routing: experts of any number of rows beside empty
ones.  Whole-number layers, whose results are exact (the argument is that of
test_int4_precision_gpu.py: |h| <= 24, a <= 576, every fp32 step below 2^24)."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import Routing, moe_experts_int4, moe_route
from tests.test_int4_gpu import _Values
from tests.test_int4_precision_gpu import _whole_codes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, I = 128, 256


def _x(n, g):
    x = torch.zeros(n, H)
    for t in range(n):
        x[t, torch.randperm(H, generator=g)[:3]] = torch.randint(0, 2, (3,), generator=g) * 2. - 1
    return x.to(torch.bfloat16)


def _check(x, idx, w, w13, w2, routing):
    out = moe_experts_int4(x.to(DEV), *w13, *w2, routing, "relu2")
    want = oracle.moe_ffn(x, idx, w, _Values(w13), _Values(w2), "relu2", "packed", {})
    assert np.abs(want).max() < 2 ** 24
    same = out.cpu() == torch.from_numpy(want).to(torch.bfloat16)
    assert bool(same.all()), f"{int((~same).sum())} of {same.numel()} values off"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n", [2, 4, 5, 7, 8, 9, 15, 16, 17, 24, 25, 33, 50])
def test_one_expert_takes_every_token(n, group):
    """Expert 3 has n rows, the others share n more: passes of 4, 8 and 16 rows."""
    print(f"[int4-rows] n={n} G={group}", flush=True)
    e, k = 40, 2
    g = torch.Generator().manual_seed(n * 1000 + group)
    lg = torch.full((n, e), -50.0)
    lg[:, 3] = 0.0
    other = torch.randint(4, e, (n,), generator=g)
    lg[torch.arange(n), other] = 0.0
    w13 = _whole_codes(g, e, I, H, group, True)
    w2 = _whole_codes(g, e, H, I, group, False)
    r = moe_route(lg.to(torch.bfloat16).to(DEV), k)
    assert int(r.col_sum[3]) == n and int(r.col_sum[0]) == 0
    _check(_x(n, g), r.topk_idx.cpu().numpy(), r.topk_w.double().cpu().numpy(), w13, w2, r)


def _routing_of(idx, e):
    """Routing metadata for chosen experts idx [N, k] with equal weights."""
    n, k = idx.shape
    flat = idx.reshape(-1)
    col = torch.sort(flat, stable=True)[1]
    row = torch.empty_like(col)
    row[col] = torch.arange(n * k)
    count = torch.bincount(flat, minlength=e)
    bits = torch.zeros(n, (e + 31) // 32, dtype=torch.int64)
    for t in range(n):
        for j in set(idx[t].tolist()):
            bits[t, j // 32] |= 1 << (j % 32)
    w = torch.full((n, k), 1.0 / k)
    i32 = {"topk_idx": idx, "bitmatrix": torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits),
           "col_sum": count, "offsets": torch.cat([count.new_zeros(1), count.cumsum(0)]),
           "col_sorted": col, "row_sorted": row}
    return Routing(**{f: v.int().to(DEV) for f, v in i32.items()}, topk_w=w.to(DEV),
                   gate_scal=w.reshape(-1).to(DEV))


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("n,k,picks", [(1, 4, [2, 2, 5, 2]), (1, 2, [0, 0]), (1, 8, [1] * 8),
                                       (2, 8, [3, 3, 3, 3, 3, 0, 3, 3]), (3, 4, [6, 1, 6, 1])])
def test_one_expert_in_several_slots_of_a_token(n, k, picks, group):
    """A routing of the caller's own may name an expert in several slots of a token:
    every slot counts, also where one token has a kernel of its own."""
    print(f"[int4-rows] n={n} {picks} G={group}", flush=True)
    e = 8
    g = torch.Generator().manual_seed(n + k)
    idx = torch.tensor([picks] * n)
    w13 = _whole_codes(g, e, I, H, group, False)
    w2 = _whole_codes(g, e, H, I, group, True)
    r = _routing_of(idx, e)
    _check(_x(n, g), idx.numpy(), r.topk_w.double().cpu().numpy(), w13, w2, r)
