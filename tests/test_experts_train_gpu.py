"""The expert FFN's forward pass that keeps its products, and its gradient, on the
GPU against the float64 oracle.

Tolerances are summed up along the computation, element by element.  u = eps / 2
of the layer dtype (half a step), U32 = 2^-24.  A sum of L fp32 products is off
by at most 2 (L + 1) U32 times the sum of its terms' magnitudes (the matrix
instructions may cut off rather than round: a whole step each), errors of the
factors enter with the other factor's magnitude, and each value that is kept in
the layer dtype adds u times its own.  The activation and its derivatives come
from the hardware's exp2 and reciprocal (a step each) of an argument alpha g that
carries up to two roundings: (16 + 8 |alpha g|) U32 of the product of their
factors' magnitudes."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import (Routing, moe_experts, moe_experts_backward,
                                        moe_experts_backward_workspace_bytes, moe_experts_ep,
                                        moe_experts_train, moe_route, moe_route_ep,
                                        prepare_experts_backward, prepare_experts_train)
from routing_grouped_expert_amd.synth import routing_logits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24
OAI = {"alpha": 1.702, "beta": 1.0, "limit": 1.5}

CASES = [
    # (N, H, I, E, k, dtype, weights, act, layout, params, zipf)
    (1, 8, 8, 1, 1, "bf16", "bf16", "silu", "packed", {}, None),
    (1, 8, 8, 1, 1, "f32", "f32", "relu2", "packed", {}, None),
    (1, 136, 72, 4, 2, "bf16", "f32", "swiglu_oai", "interleaved", OAI, None),
    (3, 64, 16, 16, 16, "f32", "f32", "silu", "interleaved", {"limit": 0.5}, None),
    (33, 128, 256, 8, 2, "f32", "f32", "silu", "packed", {}, None),
    (33, 128, 256, 8, 2, "bf16", "bf16", "silu", "packed", {}, None),
    (65, 200, 104, 5, 3, "bf16", "f32", "relu2", "packed", {}, None),
    (300, 264, 136, 3, 2, "f32", "bf16", "swiglu_oai", "packed", OAI, 1.5),
    (300, 264, 136, 3, 2, "bf16", "bf16", "swiglu_oai", "interleaved", OAI, 1.5),
    (700, 520, 392, 2, 2, "bf16", "bf16", "silu", "packed", {}, None),
    (1000, 328, 1032, 2, 1, "bf16", "f32", "silu", "interleaved", {}, None),
    (1000, 1032, 328, 4, 1, "f32", "f32", "silu", "packed", {}, None),
    (2000, 776, 520, 40, 4, "bf16", "bf16", "silu", "packed", {}, 1.1),
    (600, 2056, 2312, 4, 2, "bf16", "bf16", "swiglu_oai", "interleaved", OAI, None),
    (1500, 2304, 1288, 2, 2, "f32", "f32", "silu", "packed", {}, None),
    (40, 72, 264, 256, 4, "bf16", "bf16", "silu", "packed", {}, None),
    # row tiles of 256 rows (they have to cover the compute units)
    (4000, 2120, 2072, 3, 2, "bf16", "bf16", "swiglu_oai", "interleaved", OAI, 0.5),
    (8200, 1048, 4104, 1, 1, "bf16", "f32", "relu2", "packed", {}, None),
    (5000, 1160, 4104, 2, 1, "f32", "f32", "silu", "packed", {}, None),
    # fp32 row tiles of 64 rows: 60 and 140 rows an expert
    (320, 1160, 1096, 16, 3, "f32", "f32", "swiglu_oai", "interleaved", OAI, None),
    (420, 1672, 1608, 6, 2, "f32", "bf16", "relu2", "packed", {}, 0.5),
]


def _np(t):
    return t.detach().double().cpu().numpy()


def layer(n, h, i, e, k, dtype, weights, act, layout, params, zipf, seed=0, share=None):
    """(routing, x, d_out, w13, w2, local expert ids, sorted rows)."""
    lg = routing_logits(n, e, weights, seed=seed, zipf_s=zipf).to(DEV)
    if share is None:
        r = moe_route(lg, k)
        idx = r.topk_idx.cpu().numpy()
    else:
        r = moe_route_ep(lg, k, *share)
        idx = r.topk_idx.cpu().numpy() - share[0]
        idx = np.where((idx >= 0) & (idx < share[1]), idx, -1)
        e = share[1]
    g = torch.Generator().manual_seed(seed + 1)
    rows = i if act == "relu2" else 2 * i
    dt = DT[dtype]
    x = torch.randn(n, h, generator=g).to(dt)
    d = (torch.randn(n, h, generator=g) / 8).to(dt)
    w13 = (torch.randn(e, rows, h, generator=g) / h ** 0.5).to(dt)
    w2 = (torch.randn(e, h, i, generator=g) / i ** 0.5).to(dt)
    return r, x, d, w13, w2, idx, r.row_sorted.cpu().numpy().reshape(n, k)


def within(got, want, tol, what):
    got = _np(got)
    assert got.shape == want.shape, what
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {err.max():.3g} " \
                          f"({np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of its tolerance), " \
                          f"first at {tuple(np.argwhere(bad)[0])}"


def _parts(h, act, layout, params):
    """a, its derivatives joined in w13 order, and the error bounds of both."""
    if act == "relu2":
        a, (dg, _) = oracle.activation(act, h), oracle.activation_grad(act, h)
        return a, dg, 4 * U32 * a, 4 * U32 * dg
    alpha, beta = (params.get("alpha", 1.0), params.get("beta", 0.0)) if act == "swiglu_oai" \
        else (1.0, 0.0)
    lim = params.get("limit", np.inf)
    g, u = oracle.split_gate_up(h, layout)
    a, (dg, du) = oracle.activation(act, g, u, params), oracle.activation_grad(act, g, u, params)
    gc, uc = np.abs(np.minimum(g, lim)), np.minimum(np.abs(u), lim) + abs(beta)
    c = (16 + 8 * abs(alpha) * gc) * U32
    s = np.maximum(1 / (1 + np.exp(-alpha * np.minimum(g, lim))), 0)
    ea = c * gc * s * uc
    eg, eu = c * s * (1 + abs(alpha) * gc) * uc, c * gc * s
    join = oracle.join_gate_up
    return a, join(dg, du, layout), ea, join(eg, eu, layout)


def gradient_bounds(d, x, h, idx, w, row, w13, w2, act, layout, params, u):
    """Error bounds of the four gradients by the rules above."""
    b = {"d_x": np.zeros_like(x), "d_w13": np.zeros_like(w13), "d_w2": np.zeros_like(w2),
         "d_topk_w": np.zeros(w.shape)}
    x, d = np.abs(x), np.abs(d)
    hidden, inter = w2.shape[1:]
    for e in range(len(w13)):
        tok, slot = np.nonzero(idx == e)
        he, we = h[row[tok, slot]], np.abs(w[tok, slot])[:, None]
        a, da, ea, eda = (np.abs(v) for v in _parts(he, act, layout, params))
        sums = d[tok] @ np.abs(w2[e])                       # bounds |u| too
        eu = 2 * (hidden + 1) * U32 * sums
        b["d_topk_w"][tok, slot] = (eu * a + sums * ea +
                                    2 * (inter + 33) * U32 * sums * a).sum(1)
        two = (lambda v: v) if act == "relu2" else (lambda v: oracle.join_gate_up(v, v, layout))
        dh = we * two(sums) * (da + eda)
        edh = we * (two(eu) * da + two(sums) * eda) + (u + 4 * U32) * dh
        rows = dh @ np.abs(w13[e])
        erow = edh @ np.abs(w13[e]) + (2 * (len(w13[e]) + 1) * U32 + u) * rows
        np.add.at(b["d_x"], tok, erow + (u + 17 * U32) * (rows + erow))
        wa = we * (a + ea)
        ewa = we * ea + (u + 2 * U32) * wa
        s13, s2 = dh.T @ x[tok], d[tok].T @ wa
        c = 2 * (len(tok) + 1) * U32 + u
        b["d_w13"][e] = edh.T @ x[tok] + c * s13
        b["d_w2"][e] = d[tok].T @ ewa + c * s2
    return b


def check_gradient(got, d, x, h, idx, w, row, w13, w2, act, layout, params, u):
    args = (d, x, h, idx, w, row, w13, w2, act, layout, params)
    want, bound = oracle.moe_ffn_grad(*args), gradient_bounds(*args, u)
    for name in ("d_topk_w", "d_x", "d_w2", "d_w13"):
        within(getattr(got, name), want[name], bound[name], name)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:9])))
def test_forward_and_gradient(case):
    n, hidden, inter, e, k, dtype, weights, act, layout, params, zipf = case
    r, x, d, w13, w2, idx, row = layer(*case)
    xg, dg, w13g, w2g = (t.to(DEV) for t in (x, d, w13, w2))
    out, h = moe_experts_train(xg, w13g, w2g, r, act, layout, params)
    u = torch.finfo(DT[dtype]).eps / 2
    xn, dn, w13n, w2n, w = _np(x), _np(d), _np(w13), _np(w2), _np(r.topk_w)
    want, terms = np.zeros((n * k, len(w13n[0]))), np.zeros((n * k, len(w13n[0])))
    for i in range(e):
        tok, slot = np.nonzero(idx == i)
        want[row[tok, slot]] = xn[tok] @ w13n[i].T
        terms[row[tok, slot]] = np.abs(xn[tok]) @ np.abs(w13n[i]).T
    within(h, want, (2 * (hidden + 1) * U32 + u) * terms, "h")
    ref = oracle.moe_ffn(x, idx, w, w13, w2, act, layout, params)
    scale = np.abs(ref).max()
    assert np.abs(_np(out) - ref).max() <= (1e-4 * scale if dtype == "f32" else
                                            3e-2 + 3e-2 * scale)
    got = moe_experts_backward(dg, xg, h, w13g, w2g, r, act, layout, params)
    check_gradient(got, dn, xn, _np(h), idx, w, row, w13n, w2n, act, layout, params, u)


def _layer_on_gpu(case, **kw):
    r, x, d, w13, w2, idx, row = layer(*case, **kw)
    return r, idx, row, [t.to(DEV) for t in (x, d, w13, w2)]


SMALL = (33, 128, 72, 6, 3, "bf16", "f32", "swiglu_oai", "interleaved", OAI, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k,share", [(3, (2, 3)), (3, (5, 1)), (1, (1, 2)), (6, (0, 2))])
def test_expert_share(dtype, k, share):
    case = (70, 136, 72, 6, k, dtype, "f32", "silu", "packed", {}, 0.5)
    r, idx, row, (x, d, w13, w2) = _layer_on_gpu(case, share=share)
    n, hidden = x.shape
    routed = int(r.offsets[-1])
    fill = torch.full((n * k, w13.shape[1]), 7.0, dtype=x.dtype, device=DEV)
    out, h = moe_experts_train(x, w13, w2, r, "silu", h=fill.clone())
    assert torch.equal(h[routed:], fill[routed:])  # rows past the routed ones stay
    ref = oracle.moe_ffn(_np(x), idx, _np(r.topk_w), _np(w13), _np(w2), "silu")
    assert np.abs(_np(out) - ref).max() <= (1e-4 if dtype == "f32" else 6e-2) * np.abs(ref).max()
    assert not out[torch.from_numpy((idx < 0).all(1)).to(DEV)].any()
    h[routed:] = float("nan")  # and are not read
    got = moe_experts_backward(d, x, h, w13, w2, r, "silu")
    hn = np.nan_to_num(_np(h))
    check_gradient(got, _np(d), _np(x), hn, idx, _np(r.topk_w), row, _np(w13), _np(w2), "silu",
                   "packed", {}, torch.finfo(DT[dtype]).eps / 2)
    assert not got.d_topk_w[torch.from_numpy(idx < 0).to(DEV)].any()


def test_experts_without_rows_get_zeros_and_no_tokens_give_zeros():
    case = (3, 64, 40, 32, 2, "bf16", "bf16", "silu", "packed", {}, 1.5)
    r, idx, row, (x, d, w13, w2) = _layer_on_gpu(case)
    out, h = moe_experts_train(x, w13, w2, r, "silu")
    dirty = [torch.full_like(w, float("nan")) for w in (w13, w2)]
    got = moe_experts_backward(d, x, h, w13, w2, r, "silu", d_w13=dirty[0], d_w2=dirty[1])
    unused = [e for e in range(32) if e not in set(idx.reshape(-1).tolist())]
    assert unused and not got.d_w13[unused].any() and not got.d_w2[unused].any()
    assert torch.isfinite(got.d_w13).all() and torch.isfinite(got.d_w2).all()
    empty = Routing.empty(0, 32, 2, torch.bfloat16, DEV)
    x0, h0 = x[:0], h[:0]
    out, h = moe_experts_train(x0, w13, w2, empty, "silu")
    assert tuple(out.shape) == (0, 64) and tuple(h.shape) == (0, 80)
    got = moe_experts_backward(x0, x0, h0, w13, w2, empty, "silu",
                               d_w13=torch.full_like(w13, 3.0), d_w2=torch.full_like(w2, 3.0))
    assert not got.d_w13.any() and not got.d_w2.any() and got.d_x.numel() == 0


def test_infinities_and_nan_stay_with_their_token_and_its_experts():
    case = (64, 128, 72, 16, 2, "bf16", "bf16", "silu", "packed", {}, None)
    r, idx, row, (x, d, w13, w2) = _layer_on_gpu(case)
    clean_out, h = moe_experts_train(x, w13, w2, r, "silu")
    clean = moe_experts_backward(d, x, h, w13, w2, r, "silu")
    x2, d2 = x.clone(), d.clone()
    x2[5, 3], x2[9, 1], d2[21, 7] = float("nan"), float("inf"), float("-inf")
    out, h2 = moe_experts_train(x2, w13, w2, r, "silu")
    bad = [5, 9]
    rest = [t for t in range(64) if t not in bad]
    assert torch.equal(out[rest], clean_out[rest]) and not torch.isfinite(out[bad]).all(1).any()
    got = moe_experts_backward(d2, x2, h2, w13, w2, r, "silu")
    rest = [t for t in range(64) if t not in (5, 9, 21)]
    assert torch.equal(got.d_x[rest], clean.d_x[rest])
    assert torch.equal(got.d_topk_w[rest], clean.d_topk_w[rest])
    touched = set(idx[[5, 9, 21]].reshape(-1).tolist())
    keep = [e for e in range(16) if e not in touched]
    assert keep and torch.equal(got.d_w13[keep], clean.d_w13[keep])
    assert torch.equal(got.d_w2[keep], clean.d_w2[keep])


def test_clamp_borders():
    """Products exactly at the limit pass a gradient, those beyond pass none."""
    case = (4, 8, 8, 1, 1, "f32", "f32", "swiglu_oai", "interleaved", {}, None)
    r, idx, row, (x, d, w13, w2) = _layer_on_gpu(case)
    params = {"alpha": 1.25, "beta": 0.5, "limit": 2.0}
    h = torch.tensor([[2.0, 2.0, 2.0, -2.0, 2.25, 1.0, 1.0, 2.25, -50.0, -2.25, 0.0, 0.0,
                       -2.0, 0.5, 100.0, -100.0]] * 4, device=DEV)
    got = moe_experts_backward(d, x, h, w13, w2, r, "swiglu_oai", "interleaved", params)
    check_gradient(got, _np(d), _np(x), _np(h), idx, _np(r.topk_w), row, _np(w13), _np(w2),
                   "swiglu_oai", "interleaved", params, U32)


def test_gradient_of_the_call_itself_by_differences():
    """moe_experts_backward against central differences of moe_experts_train (fp32)."""
    case = (5, 16, 8, 3, 2, "f32", "f32", "silu", "packed", {}, None)
    r, idx, row, (x, d, w13, w2) = _layer_on_gpu(case)
    _, h = moe_experts_train(x, w13, w2, r, "silu")
    got = moe_experts_backward(d, x, h, w13, w2, r, "silu")

    def total():
        return float((moe_experts_train(x, w13, w2, r, "silu")[0].double() * d.double()).sum())
    g = torch.Generator().manual_seed(3)
    for t, grad in ((x, got.d_x), (w13, got.d_w13), (w2, got.d_w2)):
        v = torch.randn(t.shape, generator=g).to(DEV)
        step = 2.0 ** -7
        keep = t.clone()
        t.copy_(keep + step * v)
        up = total()
        t.copy_(keep - step * v)
        down = total()
        t.copy_(keep)
        want = float((grad.double() * v.double()).sum())
        # truncation: step^2 / 6 of third derivatives of O(|v|^3); rounding: 2^-24 of sums of
        # O(100) over the step
        assert abs((up - down) / (2 * step) - want) <= 2e-2 * max(1.0, abs(want))


@pytest.mark.parametrize("case", [SMALL, (600, 520, 392, 2, 2, "bf16", "bf16", "silu", "packed",
                                          {}, None)], ids=["small", "medium"])
def test_the_same_bits_prepared_on_another_stream_and_replayed(case):
    act, layout, params = case[7:10]
    r, idx, row, (x, d, w13, w2) = _layer_on_gpu(case)
    n, hidden = x.shape
    k, inter = r.topk, w2.shape[2]
    out, h = moe_experts_train(x, w13, w2, r, act, layout, params)
    want = moe_experts_backward(d, x, h, w13, w2, r, act, layout, params)

    def same(a, b):
        assert torch.equal(a[0], out) and torch.equal(a[1], h)
        for f in ("d_x", "d_w13", "d_w2", "d_topk_w"):
            assert torch.equal(getattr(b, f), getattr(want, f)), f
    fwd = prepare_experts_train(x, w13, w2, r, act, layout, params)
    bwd = prepare_experts_backward(d, x, h, w13, w2, r, act, layout, params)
    for _ in range(2):
        a, b = fwd(), bwd()
        same(a, b)
    # two calls at once on two streams, each with a workspace of its own
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    res = [(moe_experts_train(x, w13, w2, r, act, layout, params, stream=s),
            moe_experts_backward(d, x, h, w13, w2, r, act, layout, params, stream=s))
           for s in streams]
    torch.cuda.synchronize()
    for a, b in res:
        same(a, b)
    # captured with given buffers; what the workspace held does not matter
    ws = torch.empty(moe_experts_backward_workspace_bytes(n, k, hidden, inter, x.dtype),
                     dtype=torch.uint8, device=DEV)
    o2, h2 = torch.empty_like(out), torch.empty_like(h)
    b2 = type(want)(*(torch.empty_like(t) for t in (want.d_x, want.d_w13, want.d_w2,
                                                    want.d_topk_w)))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        moe_experts_train(x, w13, w2, r, act, layout, params, out=o2, h=h2)
        moe_experts_backward(d, x, h2, w13, w2, r, act, layout, params, d_x=b2.d_x,
                             d_w13=b2.d_w13, d_w2=b2.d_w2, d_topk_w=b2.d_topk_w, workspace=ws)
    for fill in (0, 255, 17):
        ws.fill_(fill)
        for t in (o2, h2, b2.d_x, b2.d_w13, b2.d_w2, b2.d_topk_w):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same((o2, h2), b2)


def test_forward_is_that_of_moe_experts():
    for case in (SMALL, (300, 264, 136, 3, 2, "f32", "f32", "silu", "packed", {}, None)):
        act, layout, params = case[7:10]
        r, idx, row, (x, d, w13, w2) = _layer_on_gpu(case)
        want = moe_experts(x, w13, w2, r, act, layout, params)
        out, _ = moe_experts_train(x, w13, w2, r, act, layout, params)
        # the same roundings (activation rows, expert rows, output) of sums in another
        # order: a half step of each may fall the other way
        scale = float(want.abs().max())
        assert float((out.float() - want.float()).abs().max()) <= \
            (1e-5 if case[5] == "f32" else 4 * 2.0 ** -8) * scale


def test_refusals():
    r, idx, row, (x, d, w13, w2) = _layer_on_gpu(SMALL)
    act, layout, params = SMALL[7:10]
    out, h = moe_experts_train(x, w13, w2, r, act, layout, params)
    ok = (d, x, h, w13, w2, r, act, layout, params)

    def swapped(i, v):
        return ok[:i] + (v,) + ok[i + 1:]
    for bad in (swapped(0, d[:-1]), swapped(0, d.float()), swapped(1, x.cpu()),
                swapped(2, h[:, :-8]), swapped(2, h.t().contiguous().t()),
                swapped(3, w13[:, :-8].contiguous()), swapped(4, w2[:-1].contiguous()),
                swapped(6, "gelu"), swapped(7, "columns"), swapped(8, {"gamma": 1.0})):
        with pytest.raises((ValueError, TypeError)):
            moe_experts_backward(*bad)
    other = moe_route(routing_logits(34, 6, "f32").to(DEV), 3)
    with pytest.raises(ValueError):
        moe_experts_backward(*swapped(5, other))
    with pytest.raises(ValueError):
        moe_experts_train(x, w13, w2, r, act, layout, params, h=h[:-1])
    with pytest.raises(Exception):
        moe_experts_backward(*ok, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
