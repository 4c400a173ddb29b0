"""Routings of expert shares where a call takes the whole layer's, and the other way
round."""
import pytest
import torch

from routing_grouped_expert_amd import (Routing, moe_experts_int4, moe_forward_ep, moe_gate_route,
                                        moe_quantize_int4, moe_route, moe_route_backward,
                                        moe_route_ep, prepare_experts_int4, prepare_route_backward)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _layer(n, e, k, h=64, i=64):
    g = torch.Generator().manual_seed(n)
    bf = {"dtype": torch.bfloat16, "device": DEV}
    x = torch.randn(n, h, generator=g).to(**bf)
    lg = torch.randn(n, e, generator=g).to(**bf)
    w13 = (torch.randn(e, 2 * i, h, generator=g) / 8).to(**bf)
    w2 = (torch.randn(e, h, i, generator=g) / 8).to(**bf)
    return x, lg, w13, w2


@pytest.mark.parametrize("n,k", [(1, 1), (20, 1), (20, 2)])
def test_4_bit_experts_refuse_the_routing_of_a_share(n, k):
    """Its rows of tokens that are routed elsewhere would be left unwritten."""
    x, lg, w13, w2 = _layer(n, 8, k)
    q13, q2 = moe_quantize_int4(w13[2:5].contiguous(), 32), moe_quantize_int4(w2[2:5].contiguous(),
                                                                              32)
    r = moe_route_ep(lg, k, 2, 3)
    assert r.layer_experts == 8
    for call in (moe_experts_int4, prepare_experts_int4):
        with pytest.raises(ValueError, match="share"):
            call(x, *q13, *q2, r, "silu")
    copy = Routing(**vars(r))
    with pytest.raises(ValueError, match="share"):
        moe_experts_int4(x, *q13, *q2, copy, "silu")
    _, r2 = moe_forward_ep(x, lg, w13[2:5].contiguous(), w2[2:5].contiguous(), k, 2, "silu")
    with pytest.raises(ValueError, match="share"):
        moe_experts_int4(x, *q13, *q2, r2, "silu")


def test_a_routing_that_is_filled_again_is_what_its_last_call_made_it():
    x, lg, w13, w2 = _layer(16, 4, 2)
    q13, q2 = moe_quantize_int4(w13, 32), moe_quantize_int4(w2, 32)
    want = moe_experts_int4(x, *q13, *q2, moe_route(lg, 2), "silu")
    r = moe_route_ep(lg, 2, 0, 4)  # a share that is the whole layer
    assert r.layer_experts is None
    assert torch.equal(moe_experts_int4(x, *q13, *q2, r, "silu"), want)
    wide = torch.cat([lg, lg - 40], 1)
    moe_route_ep(wide.contiguous(), 2, 0, 4, routing=r)
    assert r.layer_experts == 8
    with pytest.raises(ValueError, match="share"):
        moe_experts_int4(x, *q13, *q2, r, "silu")
    moe_route(lg, 2, routing=r)
    assert torch.equal(moe_experts_int4(x, *q13, *q2, r, "silu"), want)
    moe_route_ep(wide.contiguous(), 2, 0, 4, routing=r)
    moe_gate_route(x, torch.randn(4, 64, device=DEV).to(x.dtype), 2, routing=r)
    assert r.layer_experts is None


@pytest.mark.parametrize("e,lo,nl", [(8, 2, 3), (40, 32, 8), (256, 0, 64)])
def test_softmax_gradient_of_a_share_covers_the_layer(e, lo, nl):
    """topk_idx holds the layer's expert ids, so d_logits has the layer's width; the
    share's own count would drop the gradients of every expert past it."""
    n, k = 30, 2
    g = torch.Generator().manual_seed(e)
    lg = torch.randn(n, e, generator=g).to(DEV)
    dw = torch.randn(n, k, generator=g).to(DEV)
    want = moe_route_backward(dw, moe_route(lg, k))
    r = moe_route_ep(lg, k, lo, nl)
    for got in (moe_route_backward(dw, r), moe_route_backward(dw, r, e),
                prepare_route_backward(dw, r)()):
        assert got.shape == (n, e)
        assert torch.equal(got, want)
    for wrong in (nl, e + 8):
        with pytest.raises(ValueError, match="share"):
            moe_route_backward(dw, r, wrong)
