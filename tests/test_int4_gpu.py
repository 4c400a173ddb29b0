"""4-bit expert weights with group scales on the GPU: the quantiser bit-exact
against the oracle, the expert layer against the oracle on the dequantised
weights.

Tolerance of a layer output.  A product u of the first GEMM is, per group of G
weights, a sum of 2 G exact terms (x (128 + q) and -x (128 + z)) in fp32, scaled
and added to the other groups' in four chains: off by at most (2 G + K / 4 G +
16) 2^-24 times the sum of |x| s (256 + q + z).  The activation passes that on
with its slope (1.1 |up| for the gate, |g sigmoid| <= |gate| for the up value, 2
|h| for the square) and adds 16 2^-24 of its own; the activation row is rounded
to bf16 (half a step, 2^-8).  The second product and the output likewise.  The
bound is for the worst case; independent roundings give two of 2^-8 / sqrt(3) at
most, so in the 2-norm the output is held to 2^-8 as well."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import (MoeError, Routing, moe_dequantize_int4, moe_experts,
                                        moe_experts_int4, moe_forward_int4, moe_quantize_int4,
                                        moe_route, prepare_experts_int4)
from routing_grouped_expert_amd.synth import LayerSpec, act_params, layer_spec, make_layer
from tests.gpu_util import assert_output_close, assert_routing_equal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U32, U16 = 2.0 ** -24, 2.0 ** -8
OAI = {"alpha": 1.702, "beta": 1.0, "limit": 7.0}


def _weights(e, rows, k, dt, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(e, rows, k, generator=g) * 0.02
    w[0, 0, :32] = 0.0                       # zeros only (a whole group at group 32)
    w[0, -1, -32:] = -w[0, -1, -32:].abs()   # no positive weight
    w[-1, 0, :32] = 0.01 + w[-1, 0, :32].abs()  # no negative weight
    w[-1, -1, 3] = 40.0                      # an outlier
    w[-1, 1, :32] *= 1e-30                   # tiny weights
    return w.to({"bf16": torch.bfloat16, "f32": torch.float32}[dt])


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("e,rows,k,group,dt", [(3, 40, 96, 32, "bf16"), (2, 7, 2880, 64, "bf16"),
                                               (4, 33, 256, 128, "f32"), (1, 2, 32, 32, "f32"),
                                               (2, 3, 384, 128, "bf16")])
def test_quantize_bit_exact(e, rows, k, group, dt, zeros):
    print(f"[int4-q] E={e} rows={rows} K={k} G={group} {dt} zeros={zeros}", flush=True)
    w = _weights(e, rows, k, dt, seed=e * rows + k)
    q, s, z = moe_quantize_int4(w.to(DEV), group, zeros=zeros)
    rq, rs, rz = oracle.quantize_int4(w, group, zeros)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.float().cpu().numpy().transpose(0, 2, 1), rs)
    if zeros:
        assert np.array_equal(z.cpu().numpy().transpose(0, 2, 1), rz)
    else:
        assert z is None
    got = moe_dequantize_int4(q, s, z)
    want = torch.from_numpy(oracle.dequantize_int4(rq, rs, rz, group)).to(torch.bfloat16)
    assert torch.equal(got.cpu(), want)


class _Values:
    """Dequantised weights one expert at a time (float64), for the oracle."""

    def __init__(self, w):
        q, s, z = w
        self.q, self.s = q.cpu().numpy(), s.float().cpu().numpy()
        self.z = None if z is None else z.cpu().numpy()
        self.group = 2 * q.shape[2] // s.shape[1]
        self.shape = (q.shape[0], q.shape[1], 2 * q.shape[2])

    def __getitem__(self, e):
        return oracle.dequantize_int4(self.q[e], self.s[e].T,
                                      None if self.z is None else self.z[e].T, self.group)

    def reach(self, e):
        """s (256 + q + z): the size of the terms that are summed."""
        zero = 8.0 if self.z is None else self.z[e].astype(float)
        plus = oracle.dequantize_int4(self.q[e], self.s[e].T,
                                      (-256.0 - zero * np.ones_like(self.s[e])).T, self.group)
        return plus


def _bound(x, idx, w, w13, w2, act, layout, params):
    """The layer's worst-case error as the module's docstring derives it."""
    x, w = x.double().cpu().numpy(), np.asarray(w, dtype=np.float64)
    out = np.zeros((x.shape[0], w2.shape[1]))
    g, (h, i) = w13.group, (x.shape[1], w2.shape[2])
    l1 = (2 * g + h / (4 * g) + 16) * U32
    l2 = (2 * g + i / (4 * g) + 16) * U32
    lim = params.get("limit", np.inf)
    for e in range(w13.shape[0]):
        tok, slot = np.nonzero(idx == e)
        if not len(tok):
            continue
        u, du = x[tok] @ w13[e].T, l1 * (np.abs(x[tok]) @ w13.reach(e).T)
        if act == "relu2":
            a = oracle.activation(act, u)
            da = 2 * np.abs(u) * du + du * du
        else:
            gate, up = oracle.split_gate_up(u, layout)
            dg, dup = oracle.split_gate_up(du, layout)
            a = oracle.activation(act, gate, up, params)
            upm = np.minimum(np.abs(up), lim) + abs(params.get("beta", 0.0))
            da = 1.1 * dg * (upm + dup) + np.minimum(np.abs(gate), np.maximum(lim, 0)) * dup \
                + 16 * U32 * np.abs(a)
            if np.isfinite(lim):  # a gate far below zero is not limited, but its sigmoid is 0
                da += np.maximum(np.abs(gate) - lim, 0) * dup
        da = da * (1 + U16) + U16 * np.abs(a)
        y = (np.abs(a) + da) @ w2.reach(e).T * l2 + da @ np.abs(w2[e]).T
        np.add.at(out, tok, w[tok, slot][:, None] * y * (1 + 4 * U32))
    return out


CASES = [
    # (name, N, H, I, E, k, group, zeros, act, layout, params, zipf)
    ("one-token", 1, 256, 192, 16, 4, 32, True, "swiglu_oai", "interleaved", OAI, None),
    ("one-token-packed", 1, 256, 128, 16, 4, 128, False, "silu", "packed", {}, None),
    ("smallest", 1, 32, 32, 1, 1, 32, True, "silu", "packed", {}, None),
    ("relu2", 7, 96, 160, 4, 2, 32, True, "relu2", "packed", {}, None),
    ("top1", 33, 128, 256, 8, 1, 64, False, "silu", "packed", {"limit": 3.0}, None),
    ("top16", 5, 64, 64, 16, 16, 64, True, "silu", "interleaved", {}, None),
    ("tail-96", 40, 352, 224, 8, 3, 32, True, "silu", "interleaved", {}, None),
    ("tail-64", 9, 192, 448, 8, 2, 64, False, "swiglu_oai", "packed", OAI, None),
    ("sixteen-rows", 16, 128, 128, 2, 2, 128, True, "silu", "packed", {}, None),
    ("seventeen-rows", 17, 128, 128, 2, 2, 128, True, "silu", "interleaved", {}, None),
    ("thirty-three-rows", 33, 160, 96, 3, 3, 32, False, "relu2", "packed", {}, None),
    ("skewed", 100, 256, 256, 32, 4, 128, True, "swiglu_oai", "packed", OAI, 3.0),
    ("e256", 64, 128, 128, 256, 8, 64, True, "silu", "packed", {}, None),
    ("many-rows", 300, 128, 128, 4, 2, 32, True, "silu", "interleaved", {}, None),
    ("long", 3, 4096, 1536, 8, 2, 32, True, "silu", "packed", {}, None),
    # about one row an expert: w2 and the sum over the slots in one kernel
    ("seven-slots", 9, 128, 352, 64, 7, 32, True, "silu", "packed", {}, None),
    ("sixteen-slots", 1, 160, 224, 16, 16, 32, False, "silu", "interleaved", {}, None),
    ("three-slots", 20, 128, 1024, 64, 3, 128, True, "relu2", "packed", {}, None),
    ("two-slots-long", 2, 64, 8448, 8, 2, 64, True, "silu", "packed", {}, None),
    # one token, rows longer than LDS holds at a time
    ("one-token-long", 1, 64, 33280, 4, 2, 64, True, "silu", "packed", {}, None),
    ("one-token-tail", 1, 416, 96, 8, 3, 32, False, "relu2", "packed", {}, None),
    ("long-rows", 20, 64, 4416, 2, 2, 64, False, "silu", "packed", {}, None),
]


def _layer(case):
    name, n, h, i, e, k, group, zeros, act, layout, params, zipf = case
    spec = LayerSpec(name, n_tokens=n, hidden=h, inter=i, n_experts=e, topk=k, dtype="bf16",
                     act=act, layout=layout, alpha=params.get("alpha"), beta=params.get("beta"),
                     limit=params.get("limit"), zipf_s=zipf, seed=n + 3 * h)
    layer = make_layer(spec)
    return spec, layer, moe_quantize_int4(layer.w13.to(DEV), group, zeros=zeros), \
        moe_quantize_int4(layer.w2.to(DEV), group, zeros=zeros)


def _close(out, x, idx, w, w13, w2, act, layout, params, where):
    v13, v2 = _Values(w13), _Values(w2)
    want = oracle.moe_ffn(x, idx, w, v13, v2, act, layout, params)
    got = out.double().cpu().numpy()
    err = np.abs(got - want)
    tol = _bound(x, idx, w, v13, v2, act, layout, params)
    tol = tol + U16 * (np.abs(want) + tol)
    assert (err <= tol).all(), f"{where}: {int((err > tol).sum())} values off, {err.max():.3g}"
    norm = np.linalg.norm(want)
    rel = np.linalg.norm(err) / norm if norm else 0.0
    print(f"[int4] {where}: rel {rel:.2e}, worst error / bound {np.max(err / tol):.2f}", flush=True)
    assert rel <= U16, f"{where}: relative 2-norm error {rel:.3g}"


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_layer(case):
    print(f"[int4] {case}", flush=True)
    spec, layer, w13, w2 = _layer(case)
    k, act, layout, params = spec.topk, spec.act, spec.layout, act_params(spec)
    x, lg = layer.x.to(DEV), layer.logits.to(DEV)
    out, routing = moe_forward_int4(x, lg, *w13, *w2, k, act, layout, params)
    torch.cuda.synchronize()
    assert_routing_equal(routing, oracle.route(layer.logits, k, "bf16"), spec.name)
    idx, w = routing.topk_idx.cpu().numpy(), routing.topk_w.double().cpu().numpy()
    _close(out, layer.x, idx, w, w13, w2, act, layout, params, spec.name)
    again = moe_experts_int4(x, *w13, *w2, routing, act, layout, params)
    assert torch.equal(out, again)  # and the same bits every run
    # the bf16 layer on the dequantised weights is the same layer but for the
    # rounding of the weights
    ref = moe_experts(x, moe_dequantize_int4(*w13), moe_dequantize_int4(*w2), routing, act, layout,
                      params)
    assert_output_close(out, ref.double().cpu().numpy(), spec.name)


@pytest.mark.parametrize("n", [1, 33])
def test_gptoss_sized(n):
    spec = layer_spec("gptoss", n_tokens=n, name=f"gptoss_n{n}_int4", n_experts=32)
    print(f"[int4] {spec}", flush=True)
    layer = make_layer(spec)
    w13 = moe_quantize_int4(layer.w13.to(DEV), 64)
    w2 = moe_quantize_int4(layer.w2.to(DEV), 64)
    out, r = moe_forward_int4(layer.x.to(DEV), layer.logits.to(DEV), *w13, *w2, spec.topk,
                              spec.act, spec.layout, act_params(spec))
    _close(out, layer.x, r.topk_idx.cpu().numpy(), r.topk_w.double().cpu().numpy(), w13, w2,
           spec.act, spec.layout, act_params(spec), spec.name)


def test_weights_at_the_ends_of_the_code_range():
    # codes 0 and 15 with zero points 0 and 15: the products are exact integers
    n, h, i, e, k = 3, 64, 64, 2, 1
    g = torch.Generator().manual_seed(0)

    def codes(rows, kk):
        c = torch.randint(0, 2, (e, rows, kk), generator=g, dtype=torch.uint8) * 15
        z = torch.randint(0, 2, (e, kk // 32, rows), generator=g, dtype=torch.uint8) * 15
        s = torch.full((e, kk // 32, rows), 2.0 ** -6).to(torch.bfloat16)
        return [t.to(DEV) for t in (c[..., 0::2] | (c[..., 1::2] << 4), s, z)]

    w13, w2 = codes(i, h), codes(h, i)
    x = torch.randint(-2, 3, (n, h), generator=g).to(torch.bfloat16)
    lg = torch.randn(n, e, generator=g).to(torch.bfloat16)
    out, r = moe_forward_int4(x.to(DEV), lg.to(DEV), *w13, *w2, k, "relu2")
    _close(out, x, r.topk_idx.cpu().numpy(), r.topk_w.double().cpu().numpy(), w13, w2, "relu2",
           "packed", {}, "ends")


def test_rows_of_non_finite_tokens_stay_apart():
    spec, layer, w13, w2 = _layer(CASES[10])
    args = (*w13, *w2, spec.topk, spec.act, spec.layout, act_params(spec))
    x = layer.x.clone()
    want, _ = moe_forward_int4(x.to(DEV), layer.logits.to(DEV), *args)
    x[5, 7] = float("nan")
    x[20] = float("nan")
    got, _ = moe_forward_int4(x.to(DEV), layer.logits.to(DEV), *args)
    keep = torch.ones(spec.n_tokens, dtype=torch.bool)
    keep[[5, 20]] = False
    assert torch.isnan(got[5]).all() and torch.isnan(got[20]).all()
    assert torch.equal(got[keep.to(DEV)], want[keep.to(DEV)])


def test_empty_batch():
    spec, layer, w13, w2 = _layer(CASES[2])
    x = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)
    out, _ = moe_forward_int4(x, torch.empty(0, 1, dtype=torch.bfloat16, device=DEV), *w13, *w2,
                              1, "silu")
    assert out.shape == (0, 32)


def test_caller_supplied_weights_and_fp32_routing():
    # routing weights of another dtype, changed by the caller: gate_scal is what is read
    spec, layer, w13, w2 = _layer(CASES[4])
    r = moe_route(layer.logits.float().to(DEV), spec.topk)
    r.topk_w.mul_(0.37)
    r.gate_scal.copy_(r.topk_w.reshape(-1)[r.col_sorted.long()])
    out = moe_experts_int4(layer.x.to(DEV), *w13, *w2, r, spec.act, spec.layout, act_params(spec))
    _close(out, layer.x, r.topk_idx.cpu().numpy(), r.topk_w.double().cpu().numpy(), w13, w2,
           spec.act, spec.layout, act_params(spec), "fp32 routing")


def test_captured_decode_step_replays_like_eager():
    spec, layer, w13, w2 = _layer(CASES[11])
    args = (*w13, *w2, spec.topk, spec.act, spec.layout, act_params(spec))
    x, lg = layer.x.to(DEV), layer.logits.to(DEV)
    out = torch.empty_like(x)
    r = Routing.empty(spec.n_tokens, spec.n_experts, spec.topk, torch.bfloat16, DEV)
    moe_forward_int4(x, lg, *args, out=out, routing=r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe_forward_int4(x, lg, *args, out=out, routing=r)
    for rep in range(4):
        g = torch.Generator().manual_seed(rep)
        x.copy_(torch.randn(x.shape, generator=g).to(x.dtype))
        lg.copy_(torch.randn(lg.shape, generator=g).to(lg.dtype))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = moe_forward_int4(x, lg, *args)
        assert torch.equal(out, want), rep


def test_on_another_stream():
    spec, layer, w13, w2 = _layer(CASES[6])
    args = (*w13, *w2, spec.topk, spec.act, spec.layout, act_params(spec))
    x, lg = layer.x.to(DEV), layer.logits.to(DEV)
    want, _ = moe_forward_int4(x, lg, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = moe_forward_int4(x, lg, *args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    spec, layer, w13, w2 = _layer(CASES[0])
    x = layer.x.to(DEV)
    r = moe_route(layer.logits.to(DEV), spec.topk)

    def call(x=x, w13=w13, w2=w2, act=spec.act, layout=spec.layout, **kw):
        return moe_experts_int4(x, *w13, *w2, r, act, layout, OAI, **kw)

    with pytest.raises(TypeError):
        call(x=x.float())
    with pytest.raises(TypeError):
        call(w13=(w13[0], w13[1].float(), w13[2]))
    with pytest.raises(ValueError):  # another group size than w13's
        call(w2=moe_quantize_int4(layer.w2.to(DEV), 64))
    with pytest.raises(ValueError):
        call(w13=(w13[0], w13[1], w13[2][:, :1].contiguous()))
    with pytest.raises(ValueError):
        call(w13=w2)
    with pytest.raises(ValueError):
        call(act="gelu")
    with pytest.raises(ValueError):
        call(layout="rows")
    with pytest.raises(ValueError):
        call(out=torch.empty(2, 256, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(MoeError):
        call(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):  # not contiguous
        call(w13=(w13[0].transpose(0, 1), w13[1], w13[2]))
    with pytest.raises(ValueError):
        moe_quantize_int4(layer.w13.to(DEV), 48)
    with pytest.raises(ValueError):
        moe_quantize_int4(torch.zeros(1, 4, 96, device=DEV), 64)
    assert prepare_experts_int4(x, *w13, *w2, r, spec.act, spec.layout, OAI)().shape == x.shape
