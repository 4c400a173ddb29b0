"""What the 4-bit expert layer keeps between its two products: the activation rows
hold 16 bits of mantissa, so a call's one rounding to bf16 is that of its output.

Exact cases.  Scales are 1, codes and zero points give weights of -8 .. 8, a
token has at most three entries of -1 or 1, so |h| <= 24 and the squared
rectifier gives whole numbers up to 576: ten bits, which one bf16 (eight) cannot
hold and two parts can.  A group's sum of at most 128 of them times codes of up
to 143 stays below 576 * 143 * 128 = 1.06e7 < 2^24, so does the sum over K = 256
of 576 * 8 * 256 = 1.2e6, and routing weights of equal logits are powers of two:
every fp32 step is exact and the output is the whole-number result rounded once.

Gated layers.  The output's rounding is the whole error but for d, the fp32
rounding ahead of it.  Whatever d, |out - want| <= |bf16(want) - want| + 2 |d|.
In the 2-norm d is of the size of the root of the number of fp32 steps (K / G
groups of up to 4 G sums, about 4 K of them) times 2^-24 of a group's running sum
(at most G / 2 * 136 s |a| on average), against an output of about sqrt(K) * 4 s
|a|: d / out = 2 * 17 * G * 2^-24 = 2.6e-4 at most for G = 128.  The rounding
itself is at least 2^-9 / sqrt(3) = 1.1e-3 of it (half a step relative to the
value is between 2^-9 and 2^-8, its mean square a third), so 2 |d| is less than
half of it even if all errors of d pointed one way; they are independent of the
rounding, and sqrt(1 + (2.6e-4 / 1.1e-3)^2) = 1.03.  Held to 1.1.  A rounding of
the activation rows to bf16 adds as much as the output's: 1.3 to 1.4."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import moe_forward_int4, moe_quantize_int4
from routing_grouped_expert_amd.synth import LayerSpec, act_params, make_layer
from tests.test_int4_gpu import _Values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _whole_codes(g, e, rows, k, group, zeros):
    q = torch.randint(0, 256, (e, rows, k // 2), generator=g, dtype=torch.uint8)
    s = torch.ones(e, k // group, rows, dtype=torch.bfloat16)
    z = torch.randint(7, 9, s.shape, generator=g, dtype=torch.uint8) if zeros else None
    return tuple(None if t is None else t.to(DEV) for t in (q, s, z))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,e,k", [(1, 4, 1), (1, 4, 2), (3, 8, 4), (33, 16, 1), (40, 4, 2)])
def test_whole_numbers_come_through_exactly(n, e, k, group):
    print(f"[int4-exact] n={n} E={e} k={k} G={group}", flush=True)
    h, i = 128, 256
    g = torch.Generator().manual_seed(100 * n + group)
    w13 = _whole_codes(g, e, i, h, group, True)
    w2 = _whole_codes(g, e, h, i, group, n % 2 == 0)
    x = torch.zeros(n, h)
    for t in range(n):
        x[t, torch.randperm(h, generator=g)[:3]] = torch.randint(0, 2, (3,), generator=g) * 2. - 1
    x = x.to(torch.bfloat16)
    # the k selected experts have equal logits: weights 1 / k, a power of two
    lg = torch.full((n, e), -50.0)
    for t in range(n):
        lg[t, torch.randperm(e, generator=g)[:k]] = 0.0
    out, r = moe_forward_int4(x.to(DEV), lg.to(torch.bfloat16).to(DEV), *w13, *w2, k, "relu2")
    w = r.topk_w.double().cpu().numpy()
    assert (w == 1.0 / k).all()
    want = oracle.moe_ffn(x, r.topk_idx.cpu().numpy(), w, _Values(w13), _Values(w2), "relu2",
                          "packed", {})
    assert np.abs(want).max() < 2 ** 24 and np.abs(want).max() > 2 ** 9
    same = out.cpu() == torch.from_numpy(want).to(torch.bfloat16)
    assert bool(same.all()), f"{int((~same).sum())} of {same.numel()} values off"


@pytest.mark.parametrize("n,h,i,e,k,group,act,layout", [
    (1, 1024, 1536, 8, 4, 128, "silu", "packed"),
    (4, 512, 1024, 16, 2, 32, "swiglu_oai", "interleaved"),
    (60, 512, 768, 4, 2, 64, "silu", "interleaved"),
    (33, 768, 2176, 8, 1, 128, "silu", "packed"),
])
def test_error_is_that_of_one_rounding(n, h, i, e, k, group, act, layout):
    print(f"[int4-round] n={n} H={h} I={i} E={e} k={k} G={group} {act}", flush=True)
    spec = LayerSpec("p", n_tokens=n, hidden=h, inter=i, n_experts=e, topk=k, dtype="bf16",
                     act=act, layout=layout, alpha=1.702 if act == "swiglu_oai" else None, seed=n)
    layer, p = make_layer(spec), act_params(spec)
    w13 = moe_quantize_int4(layer.w13.to(DEV), group)
    w2 = moe_quantize_int4(layer.w2.to(DEV), group)
    out, r = moe_forward_int4(layer.x.to(DEV), layer.logits.to(DEV), *w13, *w2, k, act, layout, p)
    want = oracle.moe_ffn(layer.x, r.topk_idx.cpu().numpy(), r.topk_w.double().cpu().numpy(),
                          _Values(w13), _Values(w2), act, layout, p)
    err = np.linalg.norm(out.double().cpu().numpy() - want)
    once = np.linalg.norm(torch.from_numpy(want).to(torch.bfloat16).double().numpy() - want)
    print(f"[int4-round] error / one rounding's {err / once:.3f}", flush=True)
    assert err <= 1.1 * once
