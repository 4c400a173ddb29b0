"""The operators around the layer as they are used together: a whole block, a
decoding step with 4-bit experts, a training step with expert products of the
caller's own."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import (MoeError, Routing, moe_block_forward, moe_block_norm,
                                        moe_block_norm_backward, moe_combine, moe_combine_weighted,
                                        moe_combine_weighted_backward, moe_dispatch,
                                        moe_experts_int4, moe_gate_forward, moe_gate_route,
                                        moe_quantize_int4, moe_route, moe_route_backward,
                                        prepare_block_forward)
from routing_grouped_expert_amd.synth import LayerSpec, act_params, make_layer, router_inputs
from tests.gpu_util import assert_output_close

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32 = 2.0 ** -24


def _block(spec, gate, seed):
    layer = make_layer(spec)
    _, wg = router_inputs(spec.n_tokens, spec.n_experts, spec.hidden, spec.dtype, seed=seed)
    g = torch.Generator().manual_seed(seed)
    dt = layer.x.dtype
    n, h = layer.x.shape

    def rnd(*shape, std=0.2, mean=1.0):
        return (torch.randn(*shape, generator=g) * std + mean).to(dt).to(DEV)

    norm = {"w_pre": rnd(h), "w_post": rnd(h),
            "gate": {"none": None, "token": rnd(n, 1, std=0.5), "channel": rnd(h)}[gate]}
    return layer, wg.to(DEV), layer.w13.to(DEV), layer.w2.to(DEV), norm


CASES = [
    # (name, N, H, I, E, k, dtype, act, layout, gate)
    ("decode", 1, 256, 192, 16, 4, "bf16", "swiglu_oai", "interleaved", "none"),
    ("step", 33, 128, 256, 8, 1, "bf16", "silu", "packed", "token"),
    ("prompt", 700, 264, 128, 8, 2, "bf16", "relu2", "packed", "channel"),
    ("fp32", 130, 136, 72, 6, 3, "f32", "silu", "interleaved", "channel"),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_block_forward_is_the_chain_of_its_calls(case):
    name, n, h, i, e, k, dt, act, layout, gate = case
    print(f"[block] {case}", flush=True)
    spec = LayerSpec(name, n_tokens=n, hidden=h, inter=i, n_experts=e, topk=k, dtype=dt, act=act,
                     layout=layout, alpha=1.702 if act == "swiglu_oai" else None, seed=n)
    layer, wg, w13, w2, norm = _block(spec, gate, seed=n + 1)
    x, p = layer.x.to(DEV), act_params(spec)
    out, logits, routing = moe_block_forward(x, wg, w13, w2, k, act, layout, p, **norm,
                                             residual_scale=0.5)
    rows = moe_block_norm(x, w_pre=norm["w_pre"]).n_out
    y, lg, r = moe_gate_forward(rows, wg, w13, w2, k, act, layout, p)
    want = moe_block_norm(x, y, w_post=norm["w_post"], gate=norm["gate"], residual_scale=0.5)
    assert torch.equal(logits, lg) and torch.equal(routing.topk_idx, r.topk_idx)
    assert torch.equal(out, want.x_out)
    # against the oracle on the rows that were routed
    ref = oracle.moe_ffn(rows, r.topk_idx.cpu().numpy(), r.topk_w.double().cpu().numpy(),
                         layer.w13, layer.w2, act, layout, p)
    f = oracle.block_norm(x, ref, norm["w_post"], None, norm["gate"], scale=0.5)
    # a normed row is of the size of its weights whatever y's size: the layer's
    # tolerance relative to y is one relative to the row here
    assert_output_close(out, f["x_out"], name)
    # in place, and with buffers of the caller's own
    xi = x.clone()
    got = prepare_block_forward(xi, wg, w13, w2, k, act, layout, p, **norm, residual_scale=0.5,
                                x_out=xi, routing=Routing.empty(n, e, k, x.dtype, DEV))()
    assert got[0] is xi and torch.equal(xi, out)


def test_block_forward_refusals():
    spec = LayerSpec("b", n_tokens=8, hidden=64, inter=64, n_experts=4, topk=2, dtype="bf16")
    layer, wg, w13, w2, norm = _block(spec, "channel", 1)
    x = layer.x.to(DEV)

    def call(x=x, wg=wg, w13=w13, topk=2, layout="packed", **kw):
        return moe_block_forward(x, wg, w13, w2, topk, "silu", layout, **{**norm, **kw})

    with pytest.raises(ValueError):
        call(w_pre=None)
    with pytest.raises(ValueError):
        call(wg=wg[:3].contiguous())
    with pytest.raises(ValueError):
        call(w13=w13[:, :64].contiguous())
    with pytest.raises(ValueError):
        call(layout="rows")
    with pytest.raises(ValueError):
        call(gate=torch.ones(8, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        call(w_post=torch.ones(64, device=DEV))
    with pytest.raises(MoeError):
        call(topk=5)
    with pytest.raises(MoeError):
        call(workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(MoeError):
        call(eps=0.0)


def test_decoding_steps_with_4_bit_experts_in_a_graph():
    """Three layers: the fused norm between two blocks, the router GEMM, 4-bit
    experts; the captured chain replays like the eager one."""
    n, h, i, e, k, layers = 4, 256, 192, 16, 4, 3
    p = {"alpha": 1.702, "beta": 1.0, "limit": 7.0}
    w = []
    for l in range(layers):
        spec = LayerSpec(f"l{l}", n_tokens=n, hidden=h, inter=i, n_experts=e, topk=k,
                         dtype="bf16", act="swiglu_oai", layout="interleaved", seed=l)
        layer, wg, w13, w2, norm = _block(spec, "none", seed=10 + l)
        w.append((wg, moe_quantize_int4(w13, 32), moe_quantize_int4(w2, 32, zeros=False), norm))
    x = layer.x.to(DEV)

    def chain(x):
        rows = moe_block_norm(x, w_pre=w[0][3]["w_pre"]).n_out
        for l, (wg, w13, w2, norm) in enumerate(w):
            _, r = moe_gate_route(rows, wg, k)
            y = moe_experts_int4(rows, *w13, *w2, r, "swiglu_oai", "interleaved", p)
            s = moe_block_norm(x, y, w_post=norm["w_post"],
                               w_pre=w[l + 1][3]["w_pre"] if l + 1 < layers else None)
            x, rows = s.x_out, s.n_out
        return x

    chain(x)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(buf)
    for rep in range(4):
        g = torch.Generator().manual_seed(rep)
        buf.copy_(torch.randn(n, h, generator=g).to(buf.dtype))
        graph.replay()
        torch.cuda.synchronize()
        want = chain(buf)
        assert torch.equal(out, want), rep
        assert torch.isfinite(out).all()


def test_training_step_with_the_callers_own_experts():
    """Forward and backward through a block whose expert products are torch's:
    every gradient against float64 reverse-mode differentiation of the plain
    definition with the same selection.

    In fp32 every value is a chain of about ten sums of at most 520 terms, so
    its error is at most 10 * 520 * 2^-24 = 3.1e-4 of the sum of its terms'
    magnitudes; independent roundings stay far below that in the 2-norm."""
    n, h, i, e, k = 203, 136, 72, 6, 3
    g = torch.Generator().manual_seed(0)

    def rnd(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g) * std + mean

    p = {"x": rnd(n, h), "w_pre": rnd(h, std=0.2, mean=1), "wg": rnd(e, h, std=h ** -0.5),
         "w1": rnd(e, i, h, std=h ** -0.5), "w2": rnd(e, h, i, std=i ** -0.5),
         "w_post": rnd(h, std=0.2, mean=1), "gate": rnd(n, 1, std=0.5)}
    d_out, scale = rnd(n, h), 0.5
    q = {a: v.to(DEV) for a, v in p.items()}

    # ---- forward
    pre = moe_block_norm(q["x"], w_pre=q["w_pre"])
    logits = pre.n_out @ q["wg"].t()
    r = moe_route(logits, k)
    off = r.offsets.tolist()
    xs = moe_dispatch(pre.n_out, r)
    u = torch.empty(n * k, i, device=DEV)
    ys = torch.empty(n * k, h, device=DEV)
    for j in range(e):
        u[off[j]:off[j + 1]] = xs[off[j]:off[j + 1]] @ q["w1"][j].t()
        ys[off[j]:off[j + 1]] = torch.tanh(u[off[j]:off[j + 1]]) @ q["w2"][j].t()
    y = moe_combine_weighted(ys, r)
    post = moe_block_norm(q["x"], y, w_post=q["w_post"], gate=q["gate"], residual_scale=scale)
    # ---- backward
    b = moe_block_norm_backward(d_out.to(DEV), None, q["x"], y, w_post=q["w_post"],
                                gate=q["gate"], residual_scale=scale, rstd_post=post.rstd_post)
    d_ys, d_w = moe_combine_weighted_backward(b.d_y, ys, r)
    d_logits = moe_route_backward(d_w, r)
    got = {"w_post": b.d_w_post, "gate": b.d_gate, "w1": torch.empty_like(q["w1"]),
           "w2": torch.empty_like(q["w2"]), "wg": d_logits.t() @ pre.n_out}
    d_xs = torch.empty_like(xs)
    for j in range(e):
        s = slice(off[j], off[j + 1])
        a = torch.tanh(u[s])
        got["w2"][j] = d_ys[s].t() @ a
        du = (d_ys[s] @ q["w2"][j]) * (1 - a * a)
        got["w1"][j] = du.t() @ xs[s]
        d_xs[s] = du @ q["w1"][j]
    d_rows = moe_combine(d_xs, r) + d_logits @ q["wg"]
    f = moe_block_norm_backward(b.d_x, d_rows, q["x"], w_pre=q["w_pre"], rstd_pre=pre.rstd_pre)
    got["x"], got["w_pre"] = f.d_x, f.d_w_pre

    # ---- the plain definition in float64
    z = {a: v.double().requires_grad_() for a, v in p.items()}
    idx = r.topk_idx.long().cpu()

    def rms(v, w):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w

    rows = rms(z["x"], z["w_pre"])
    w = torch.softmax((rows @ z["wg"].t()).gather(1, idx), 1)
    yy = torch.zeros(n, h, dtype=torch.float64)
    for j in range(e):
        full = torch.tanh(rows @ z["w1"][j].t()) @ z["w2"][j].t()
        yy = yy + full * (w * (idx == j)).sum(1, keepdim=True)
    out = z["x"] + scale * z["gate"] * rms(yy, z["w_post"])
    want = dict(zip(z, torch.autograd.grad((out * d_out.double()).sum(), list(z.values()))))
    assert torch.allclose(post.x_out.double().cpu(), out.detach(), rtol=0, atol=1e-4)
    for a in p:
        err = (got[a].double().cpu() - want[a]).norm() / want[a].norm()
        print(f"[train] d_{a}: rel {err:.2e}", flush=True)
        assert err <= 3.1e-4, (a, float(err))


def test_expert_shares_add_up_to_the_layer():
    """Combine, its gradient and the softmax gradient over the shares of an
    expert-parallel group add up to the whole layer's."""
    from routing_grouped_expert_amd import moe_route_ep
    n, h, e, k = 150, 72, 8, 3
    g = torch.Generator().manual_seed(4)
    lg = torch.randn(n, e, generator=g).to(DEV)
    d = torch.randn(n, h, generator=g).to(DEV)
    x = torch.randn(n, h, generator=g).to(DEV)
    whole = moe_route(lg, k)
    # the expert's output is the row times the expert's number
    rows = moe_dispatch(x, whole)
    expert = torch.repeat_interleave(torch.arange(1, e + 1, device=DEV), whole.col_sum.long())
    y = rows * expert[:, None]
    out = moe_combine_weighted(y, whole)
    dy, dw = moe_combine_weighted_backward(d, y, whole)
    dl = moe_route_backward(dw, whole)
    o2, w2, l2 = torch.zeros_like(out), torch.zeros_like(dw), torch.zeros_like(dl)
    for lo, nl in ((0, 3), (3, 1), (4, 4)):
        r = moe_route_ep(lg, k, lo, nl)
        m = int(r.offsets[-1])
        start = int(whole.offsets[lo])
        part = torch.full((n * k, h), float("nan"), device=DEV)
        part[:m] = y[start:start + m]
        o2 += moe_combine_weighted(part, r)
        pdy, pdw = moe_combine_weighted_backward(d, part, r)
        assert torch.equal(pdy[:m], dy[start:start + m])
        w2 += pdw
        l2 += moe_route_backward(pdw, r, e)
    assert torch.equal(w2, dw)  # every slot is in one share
    mag = float(out.abs().max()) * k
    assert (o2 - out).abs().max() <= 8 * U32 * mag
    assert (l2 - dl).abs().max() <= 16 * U32 * float(dw.abs().max())
