"""A training step of a mixture-of-experts layer through the package's calls alone,
against a float64 step by torch's differentiation and the oracle's optimizer."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import (moe_adamw, moe_adamw_state, moe_experts_backward,
                                        moe_experts_train, moe_grad_norm, moe_route,
                                        moe_route_backward)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _layer64(x, logits, w13, w2, idx, k):
    """The layer in float64 with the selection given: sum of topk_w W2 silu-gated W13 x."""
    out = torch.zeros_like(x)
    w = torch.softmax(logits.gather(1, idx), 1)
    inter = w2.shape[2]
    for e in range(len(w13)):
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        h = x[tok] @ w13[e].t()
        a = torch.nn.functional.silu(h[:, :inter]) * h[:, inter:]
        out = out.index_add(0, tok, w[tok, slot][:, None] * (a @ w2[e].t()))
    return out


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_of_a_layer(bits):
    """Three steps of least squares in fp32: gradients of x, the logits and both weight
    arrays against float64, then the weights after the step against the oracle's from
    the call's own gradients."""
    n, hidden, inter, e, k = 96, 64, 40, 8, 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn(n, hidden, generator=g).to(DEV)
    logits = torch.randn(n, e, generator=g).to(DEV)
    target = torch.randn(n, hidden, generator=g).to(DEV)
    params = [(torch.randn(e, 2 * inter, hidden, generator=g) / 8).to(DEV),
              (torch.randn(e, hidden, inter, generator=g) / 8).to(DEV)]
    state = moe_adamw_state(params, bits)
    hyper = {"lr": 1e-2, "eps": 1e-8, "weight_decay": 0.1}
    for step in (1, 2, 3):
        w13, w2 = params
        routing = moe_route(logits, k)
        out, h = moe_experts_train(x, w13, w2, routing, "silu")
        d_out = (out - target) / n
        grads = moe_experts_backward(d_out, x, h, w13, w2, routing, "silu")
        d_logits = moe_route_backward(grads.d_topk_w, routing)

        leaves = [t.double().requires_grad_() for t in (x, logits, w13, w2)]
        out64 = _layer64(*leaves, routing.topk_idx.long(), k)
        want = torch.autograd.grad((out64 * d_out.double()).sum(), leaves)
        for name, got, ref in zip(("x", "logits", "w13", "w2"),
                                  (grads.d_x, d_logits, grads.d_w13, grads.d_w2), want):
            # sums of at most 192 fp32 products through four of them in a row
            err = float((got.double() - ref).abs().max() / ref.abs().max())
            assert err <= 4 * 2 * 193 * 2.0 ** -24, (step, name, err)

        before = [(p.double().cpu().numpy(), m, v) for p, m, v in
                  zip(params, *_moments(state))]
        gw = [grads.d_w13, grads.d_w2]
        norm = moe_grad_norm(gw)
        moe_adamw(params, gw, state, step=step, grad_norm=norm, max_norm=0.05, seed=step, **hyper)
        coef = oracle.clip_coefficient(float(norm), 0.05)
        for p, grad, (p0, m0, v0) in zip(params, gw, before):
            w, _, _ = oracle.adamw(p0, grad.double().cpu().numpy(), m0, v0, beta1=0.9,
                                   beta2=0.999, step=step, coef=coef, **hyper)
            # the update is at most 3 lr here and off by 2^-19 of its terms, p by its steps
            assert np.abs(p.double().cpu().numpy() - w).max() <= 1e-2 * 2.0 ** -15 + 2.0 ** -23


def _moments(state):
    if state.m_scale is None:
        return ([t.double().cpu().numpy() for t in state.m],
                [t.double().cpu().numpy() for t in state.v])

    def wide(q, s):
        return (q.float().double().reshape(-1) *
                s.double().repeat_interleave(256)[:q.numel()]).reshape(q.shape).cpu().numpy()
    return ([wide(q, s) for q, s in zip(state.m, state.m_scale)],
            [wide(q, s) ** 2 for q, s in zip(state.v, state.v_scale)])
