"""Rows into expert-sorted order and back with the routing weights, and the
gradients, on the GPU against the float64 oracle.

Tolerances.  u = eps / 2 of the output type (half a step).  A sum of L fp32
terms in any order, each product rounded or fused, is off by at most
(L + 1) 2^-24 times the sum of its terms' magnitudes; then one rounding."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import (MoeError, Routing, moe_combine, moe_combine_weighted,
                                        moe_combine_weighted_backward, moe_dispatch, moe_route,
                                        moe_route_backward, moe_route_ep, prepare_combine_weighted,
                                        prepare_combine_weighted_backward, prepare_dispatch,
                                        prepare_route_backward)
from routing_grouped_expert_amd.synth import routing_logits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24

CASES = [
    # (N, H, E, k, rows, weights)
    (1, 8, 1, 1, "bf16", "bf16"),
    (1, 2880, 128, 4, "bf16", "f32"),
    (2, 16, 16, 16, "f32", "f32"),
    (33, 128, 8, 2, "f32", "bf16"),
    (65, 136, 40, 3, "bf16", "bf16"),
    (129, 520, 7, 5, "bf16", "f32"),
    (300, 1416, 40, 6, "f32", "f32"),
    (257, 4096, 64, 8, "bf16", "bf16"),
    (31, 8200, 256, 7, "bf16", "bf16"),
    (2051, 72, 12, 9, "f32", "f32"),
    (2500, 264, 64, 8, "bf16", "bf16"),
    (5000, 64, 256, 1, "bf16", "bf16"),
]


def _inputs(n, h, e, k, rows, weights, seed=0, share=None):
    lg = routing_logits(n, e, weights, seed=seed, zipf_s=0.7).to(DEV)
    r = moe_route(lg, k) if share is None else moe_route_ep(lg, k, *share)
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(n, h, generator=g).to(DT[rows])
    y = torch.randn(n * k, h, generator=g).to(DT[rows])
    d = (torch.randn(n, h, generator=g) / 8).to(DT[rows])
    return r, x, y, d


def _half(t):
    return torch.finfo(t.dtype).eps / 2


def _np(t):
    return t.detach().double().cpu().numpy()


def _within(got, want, tol, what):
    err = np.abs(_np(got) - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {err.max():.3g}, " \
                          f"first at {tuple(np.argwhere(bad)[0])}"


def _check_all(r, x, y, d, e, k, rows_kept):
    """Every call against the oracle; rows_kept: sorted rows no slot points to."""
    n, h = x.shape
    row = r.row_sorted.cpu().numpy()
    w = _np(r.topk_w)
    fill = 7.0
    kept = torch.full((n * k, h), fill, dtype=x.dtype, device=DEV)
    xs = moe_dispatch(x.to(DEV), r, x_sorted=kept.clone())
    _within(xs, oracle.dispatch(x, row, k, into=kept), 0.0, "x_sorted")
    out = moe_combine_weighted(y.to(DEV), r)
    want = oracle.combine_weighted(y, row, w)
    terms = oracle.combine_weighted(y.abs(), row, w)
    _within(out, want, _half(out) * np.abs(want) + 2 * (k + 1) * U32 * terms, "out")
    dy, dw = moe_combine_weighted_backward(d.to(DEV), y.to(DEV), r, d_y_sorted=kept.clone())
    wdy, wdw = oracle.combine_weighted_grad(d, y, row, w, into=kept)
    _within(dy, wdy, (_half(dy) * (1 + 2 * U32) + U32) * np.abs(wdy) *
            (np.arange(n * k) < rows_kept)[:, None], "d_y_sorted")
    _, terms = oracle.combine_weighted_grad(d.abs(), y.abs(), row, w)
    _within(dw, wdw, (h + 1) * U32 * terms, "d_topk_w")
    assert not _np(dw).reshape(-1)[row < 0].any()
    # the softmax gradient from the kernel's own d_topk_w
    dl = moe_route_backward(dw, r, e)
    idx, dwn = r.topk_idx.cpu().numpy(), _np(dw)
    want = oracle.topk_weight_grad(dwn, idx, w, e)
    terms = np.zeros_like(want)
    mag = w * (np.abs(dwn) + (w * np.abs(dwn)).sum(1, keepdims=True))
    np.put_along_axis(terms, idx.astype(np.int64), mag, 1)
    _within(dl, want, _half(dl) * np.abs(want) + (k + 4) * U32 * terms, "d_logits")


@pytest.mark.parametrize("case", CASES, ids=[f"n{c[0]}h{c[1]}e{c[2]}k{c[3]}{c[4]}{c[5]}"
                                             for c in CASES])
def test_rows_against_oracle(case):
    n, h, e, k, rows, weights = case
    print(f"[rows] {case}", flush=True)
    r, x, y, d = _inputs(n, h, e, k, rows, weights, seed=n + h)
    _check_all(r, x, y, d, e, k, n * k)


@pytest.mark.parametrize("n,h,e,k,lo,nl", [(70, 136, 16, 4, 5, 6), (9, 64, 32, 3, 31, 1),
                                           (2100, 72, 8, 2, 0, 3)])
def test_share_skips_slots_and_leaves_rows(n, h, e, k, lo, nl):
    print(f"[rows-share] {n, h, e, k, lo, nl}", flush=True)
    r, x, y, d = _inputs(n, h, e, k, "bf16", "bf16", seed=n, share=(lo, nl))
    local = int(r.offsets[-1])
    assert local < n * k and (r.row_sorted < 0).any()
    y[local:] = float("nan")  # rows that no slot points to are never read
    _check_all(r, x, y, d, e, k, local)


def test_share_with_no_entries():
    # every token goes elsewhere: zero outputs and gradients, nothing moved
    n, h, e, k = 40, 64, 8, 2
    lg = torch.zeros(n, e)
    lg[:, :2] = 5.0
    r = moe_route_ep(lg.to(torch.bfloat16).to(DEV), k, 4, 3)
    x = torch.randn(n, h).to(torch.bfloat16).to(DEV)
    bad = torch.full((n * k, h), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert torch.isnan(moe_dispatch(x, r, x_sorted=bad.clone())).all()
    assert not moe_combine_weighted(bad, r).any()
    dy, dw = moe_combine_weighted_backward(x, bad, r, d_y_sorted=bad.clone())
    assert torch.isnan(dy).all() and not dw.any()
    assert not moe_route_backward(dw, r, e).any()


def test_non_finite_rows_stay_in_their_token():
    r, x, y, d = _inputs(50, 72, 8, 2, "bf16", "bf16")
    row = r.row_sorted.cpu().view(50, 2).long()
    y[row[3, 0]] = float("inf")
    y[row[20, 1], 5] = float("nan")
    out = moe_combine_weighted(y.to(DEV), r).cpu()
    bad = ~torch.isfinite(out)
    assert bad[3].all() and bad[20, 5] and bad.sum() == 73
    d[7] = float("nan")
    dy, dw = (t.cpu() for t in moe_combine_weighted_backward(d.to(DEV), y.to(DEV), r))
    rows = torch.isnan(dy).any(1).nonzero()[:, 0].tolist()
    assert sorted(rows) == sorted(row[7].tolist())
    assert torch.isfinite(dw).all(1).logical_not().nonzero()[:, 0].tolist() == [3, 7, 20]


def test_empty_batch():
    r = Routing.empty(0, 8, 2, torch.bfloat16, DEV)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert moe_dispatch(x, r).shape == (0, 64)
    assert moe_combine_weighted(x, r).shape == (0, 64)
    dy, dw = moe_combine_weighted_backward(x, x, r)
    assert dy.shape == (0, 64) and dw.shape == (0, 2)
    assert moe_route_backward(dw, r).shape == (0, 8)


def test_dispatch_gradient_is_moe_combine():
    # d_x = sum over the slots of d_x_sorted: the adjoint of the dispatch
    r, x, y, _ = _inputs(130, 264, 16, 4, "f32", "f32")
    dx = moe_combine(y.to(DEV), r)
    xs = moe_dispatch(x.to(DEV), r)
    lhs, rhs = (_np(xs) * _np(y)).sum(), (_np(x) * _np(dx)).sum()
    scale = (np.abs(_np(xs)) * np.abs(_np(y))).sum()
    assert abs(lhs - rhs) <= 6 * U32 * scale


def test_same_bits_every_run_and_on_another_stream():
    r, x, y, d = _inputs(3000, 136, 32, 4, "bf16", "bf16")
    x, y, d = x.to(DEV), y.to(DEV), d.to(DEV)

    def run(stream=None):
        xs = moe_dispatch(x, r, stream=stream)
        out = moe_combine_weighted(y, r, stream=stream)
        dy, dw = moe_combine_weighted_backward(d, y, r, stream=stream)
        return [xs, out, dy, dw, moe_route_backward(dw, r, stream=stream)]

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = run(side)
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_captured_calls_replay_like_eager_ones():
    n, h, e, k = 257, 264, 16, 4
    r, x, y, d = _inputs(n, h, e, k, "bf16", "bf16")
    x, y, d = x.to(DEV), y.to(DEV), d.to(DEV)
    # buffers made before the capture; one call twice in the graph, into one buffer
    calls = [prepare_dispatch(x, r), prepare_combine_weighted(y, r),
             prepare_combine_weighted(y, r), prepare_combine_weighted_backward(d, y, r)]
    calls.append(prepare_route_backward(calls[-1].result[1], r))
    outs = [calls[0].result, calls[1].result, *calls[3].result, calls[4].result]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s = torch.cuda.current_stream()
        graphed = [prepare_dispatch(x, r, x_sorted=outs[0], stream=s),
                   prepare_combine_weighted(y, r, out=outs[1], stream=s),
                   prepare_combine_weighted(y, r, out=outs[1], stream=s),
                   prepare_combine_weighted_backward(d, y, r, d_y_sorted=outs[2],
                                                     d_topk_w=outs[3], stream=s),
                   prepare_route_backward(outs[3], r, d_logits=outs[4], stream=s)]
        for c in graphed:
            c()
    for rep in range(4):
        g = torch.Generator().manual_seed(50 + rep)
        for t in (x, y, d):
            t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = [moe_dispatch(x, r), moe_combine_weighted(y, r),
                *moe_combine_weighted_backward(d, y, r)]
        want.append(moe_route_backward(want[3], r))
        for a, b in zip(outs, want):
            assert torch.equal(a, b), rep


def test_row_offsets_past_32_bits():
    # the sorted rows hold 2.6e9 values: element offsets pass 2^31 and byte offsets 2^32
    n, h, e, k = 20011, 8192, 64, 16
    r = moe_route(routing_logits(n, e, "bf16", seed=3).to(DEV), k)
    x = torch.randn(n, h, device=DEV, dtype=torch.bfloat16)
    xs = moe_dispatch(x, r)
    row = r.row_sorted.view(n, k).long()
    for j in (0, k - 1):
        assert torch.equal(xs[row[:, j]], x)
    out = moe_combine_weighted(xs, r)
    # every row of a token is the same: out = x * sum(w)
    want = x.float() * r.topk_w.float().sum(1, keepdim=True)
    assert (out.float() - want).abs().le(2.0 ** -8 * want.abs() + 1e-6 * x.float().abs()).all()
    dy, dw = moe_combine_weighted_backward(x, xs, r, d_y_sorted=xs.clone())
    for j in (0, k - 1):
        want = (x.float() * r.topk_w[:, j:j + 1].float()).to(torch.bfloat16)
        assert torch.equal(dy[row[:, j]], want)
    norm2 = x.double().square().sum(1)
    assert ((dw.double() - norm2[:, None]).abs() <= (h + 1) * U32 * norm2[:, None]).all()


def test_refusals():
    r, x, y, d = _inputs(20, 64, 8, 2, "bf16", "bf16")
    x, y, d = x.to(DEV), y.to(DEV), d.to(DEV)
    dw = torch.zeros(20, 2, device=DEV)
    with pytest.raises(ValueError):
        moe_dispatch(x[:19].contiguous(), r)
    with pytest.raises(ValueError):
        moe_dispatch(x.cpu(), r)
    with pytest.raises(ValueError):  # not contiguous
        moe_dispatch(x.t().contiguous().t(), r)
    with pytest.raises(TypeError):
        moe_dispatch(x.half(), r)
    with pytest.raises(ValueError):
        moe_dispatch(x, r, x_sorted=y[:39].contiguous())
    with pytest.raises(ValueError):
        moe_combine_weighted(y[:39].contiguous(), r)
    with pytest.raises(ValueError):
        moe_combine_weighted(y, r, out=torch.empty(20, 64, device=DEV))
    with pytest.raises(ValueError):
        moe_combine_weighted_backward(d[:, :56].contiguous(), y, r)
    with pytest.raises(ValueError):
        moe_combine_weighted_backward(d.float(), y, r)
    with pytest.raises(ValueError):
        moe_route_backward(dw.double(), r)
    with pytest.raises(MoeError):  # a width that is no multiple of 8
        moe_dispatch(x[:, :60].contiguous(), r)
    with pytest.raises(MoeError):  # fewer experts than slots
        moe_route_backward(dw, r, 1)
    bad = Routing(**{**vars(r), "row_sorted": r.row_sorted.long()})
    with pytest.raises(TypeError):
        moe_combine_weighted(y, bad)
    bad = Routing(**{**vars(r), "row_sorted": r.row_sorted[:39]})
    with pytest.raises(ValueError):
        moe_dispatch(x, bad)
    bad = Routing(**{**vars(r), "topk_w": r.topk_w[:, :1]})
    with pytest.raises(ValueError):
        moe_combine_weighted(y, bad)


def test_positions_out_of_range_are_skipped():
    # the documented contract: a slot outside [0, N*k) moves and adds nothing
    r, x, y, d = _inputs(12, 64, 8, 2, "f32", "f32")
    row = r.row_sorted.clone()
    row[5], row[9] = 24, 2 ** 31 - 1
    r2 = Routing(**{**vars(r), "row_sorted": row})
    want = Routing(**{**vars(r), "row_sorted": torch.where(row >= 24, -1, row).int()})
    x, y, d = x.to(DEV), y.to(DEV), d.to(DEV)
    z = torch.zeros(24, 64, device=DEV)
    assert torch.equal(moe_dispatch(x, r2, x_sorted=z.clone()),
                       moe_dispatch(x, want, x_sorted=z.clone()))
    assert torch.equal(moe_combine_weighted(y, r2), moe_combine_weighted(y, want))
    for a, b in zip(moe_combine_weighted_backward(d, y, r2, d_y_sorted=z.clone()),
                    moe_combine_weighted_backward(d, y, want, d_y_sorted=z.clone())):
        assert torch.equal(a, b)
