"""The norms around a block and their gradients on the GPU against the float64
oracle.

Tolerances.  Every value is a chain of fp32 roundings (sums included) and one
rounding to the output type.  The kernels compute sums of products, so their
error is at most L 2^-24 times the same expression with every term replaced by
its magnitude (the "terms" below), L the number of roundings on the longest
path, plus half a step of the output type.  A row sum over H values adds at most
H / 16 terms a thread (no width gives a thread of a row fewer than 1/16 of it,
and at most 32), 6 steps in the wave and up to 16 waves; a rstd takes half of
its sum's error and two more roundings (square root and division, a step each)."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import (MoeError, moe_block_norm, moe_block_norm_backward,
                                        prepare_block_norm, prepare_block_norm_backward)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24
EPS = 1e-6
ROW = 32 + 6 + 16 + 4  # roundings of one row sum, the mean and its rstd


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(n, h, dt, gate="none", branch=True, post=True, pre=True, seed=0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g) * std + mean).to(DT[dt])

    a = {"x": rnd(n, h, std=2.0), "y": rnd(n, h, std=0.7) if branch else None,
         "w_post": rnd(h, std=0.3, mean=1.0) if post else None,
         "w_pre": rnd(h, std=0.3, mean=1.0) if pre else None,
         "gate": {"none": None, "token": rnd(n, 1), "channel": rnd(h, std=0.5)}[gate]}
    d = {"d_x_out": rnd(n, h, std=0.1), "d_n_out": rnd(n, h, std=0.1) if pre else None}
    return a, d


def _dev(a):
    return {k: None if v is None else v.to(DEV) for k, v in a.items()}


def _within(got, want, terms, rounds, what):
    g = _np(got)
    assert g.shape == want.shape, f"{what}: {g.shape}"
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(g - want)
    bad = ~(err <= half * (1 + 1e-3) * np.abs(want) + rounds * U32 * terms)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {err.max():.3g}, " \
                          f"first at {tuple(np.argwhere(bad)[0])}"


def _terms(a, d, scale):
    """Every output of both directions with its terms' magnitudes (float64)."""
    m = {k: None if v is None else np.abs(_np(v)) for k, v in {**a, **d}.items()}
    f = oracle.block_norm(**a, scale=scale, eps=EPS)
    rp, rq = f["rstd_post"], f["rstd_pre"]
    t = {}
    x = m["x"]
    z = None
    g = 1.0 if m["gate"] is None else m["gate"]
    if m["y"] is not None:
        z = m["y"] if rp is None else m["y"] * rp[:, None] * m["w_post"]
        x = x + abs(scale) * g * z
        t["x_out"] = x
    dx = np.zeros_like(x) if m["d_x_out"] is None else m["d_x_out"]
    if rq is not None:
        xh = x * rq[:, None]
        # the row's x_out may be off by its terms, which moves the rstd too
        t["n_out"] = (xh + np.abs(_np(a["x"]) if f["x_out"] is None else f["x_out"])
                      * rq[:, None] * (xh * xh).mean(1, keepdims=True)) * m["w_pre"]
        g1 = m["d_n_out"] * m["w_pre"]
        t["d_w_pre"] = (m["d_n_out"] * xh).sum(0)
        dx = dx + rq[:, None] * (g1 + xh * (g1 * xh).mean(1, keepdims=True))
    t["d_x"] = dx
    if z is not None:
        sd = abs(scale) * dx
        if m["gate"] is not None:
            t["d_gate"] = (sd * z).sum(1, keepdims=True) if m["gate"].ndim == 2 \
                else (sd * z).sum(0)
        dz = sd * g
        if rp is not None:
            yh = m["y"] * rp[:, None]
            g2 = dz * m["w_post"]
            t["d_w_post"] = (dz * yh).sum(0)
            t["d_y"] = rp[:, None] * (g2 + yh * (g2 * yh).mean(1, keepdims=True))
        else:
            t["d_y"] = dz
    return f, t


def _check(a, d, scale=1.0):
    n = a["x"].shape[0]
    da, dd = _dev(a), _dev(d)
    f, t = _terms(a, d, scale)
    got = moe_block_norm(**da, residual_scale=scale, eps=EPS)
    for name in ("x_out", "n_out", "rstd_post", "rstd_pre"):
        v = getattr(got, name)
        assert (v is None) == (f[name] is None), name
        if v is None:
            continue
        terms = t[name] if name in t else np.abs(f[name])
        if name == "rstd_pre" and "x_out" in t:  # x_out's own error moves the mean
            xh = t["x_out"] * f["rstd_pre"][:, None]
            terms = terms * (1 + (xh * xh).mean(1))
        _within(v, f[name], terms, 2 * ROW, name)
    want = oracle.block_norm_grad(**d, **a, scale=scale, eps=EPS)
    g = moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, residual_scale=scale,
                                rstd_post=got.rstd_post, rstd_pre=got.rstd_pre)
    # the rstds come with their own error (up to 2 ROW, and more with x_out's
    # terms), enter twice, and two row sums follow; then the sum over the tokens
    shift = 1.0
    if "x_out" in t and f["rstd_pre"] is not None:
        xh = t["x_out"] * f["rstd_pre"][:, None]
        shift = 1 + (xh * xh).mean(1).max()
    for name in ("d_x", "d_y", "d_w_post", "d_w_pre", "d_gate"):
        v = getattr(g, name)
        assert (v is None) == (want[name] is None), name
        if v is not None:
            over_tokens = name.startswith("d_w") or (name == "d_gate" and a["gate"].dim() == 1)
            _within(v, want[name], t[name], 8 * ROW * shift + (n if over_tokens else 0), name)
    return got, g


WIDTHS = [(5, 8), (37, 64), (18, 72), (40, 128), (7, 136), (300, 512), (13, 520), (9, 1024),
          (67, 1032), (5, 2056), (35, 2880), (6, 4096), (3, 4104), (2, 8192), (3, 8200),
          (2, 16384)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,h", WIDTHS)
def test_every_width(n, h, dt):
    print(f"[norm] n={n} h={h} {dt}", flush=True)
    _check(*_inputs(n, h, dt, "channel", seed=h), scale=0.22)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gate,branch,post,pre", [
    (g, 1, post, pre) for g in ("none", "token", "channel") for post in (0, 1) for pre in (0, 1)
] + [("none", 0, 0, 1)])
@pytest.mark.parametrize("n,h", [(19, 264), (3, 1416)])
def test_every_form(n, h, gate, branch, post, pre, dt):
    print(f"[norm] n={n} h={h} {gate} {branch} {post} {pre} {dt}", flush=True)
    _check(*_inputs(n, h, dt, gate, branch, post, pre, seed=n), scale=-0.5 if branch else 1.0)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 511, 513, 2049, 8200])
def test_token_counts(n):
    print(f"[norm] n={n}", flush=True)
    _check(*_inputs(n, 256, "bf16", "token", seed=n))
    _check(*_inputs(n, 72, "f32", "channel", seed=n))


def test_gate_of_one_token_and_square_shapes():
    # [N, 1] and [hidden] stay apart where N = hidden, and where N = 1
    for n in (1, 16):
        for gate in ("token", "channel"):
            _check(*_inputs(n, 16, "f32", gate, seed=n))


def test_no_gradient_from_the_residual():
    a, d = _inputs(21, 264, "bf16", "token")
    d["d_x_out"] = None
    _check(a, d)


def test_zero_rows_and_large_values():
    a, d = _inputs(9, 128, "f32")
    a["x"][2] = 0.0
    a["y"][2] = 0.0   # a padded token: rstd = 1 / sqrt(eps), outputs zero
    a["y"][5] = 0.0
    a["x"][7] *= 1e12
    got, _ = _check(a, d)
    assert not got.x_out[2].any() and not got.n_out[2].any()
    assert float(got.rstd_post[2]) == pytest.approx(1e3, rel=1e-6)


def test_non_finite_rows_stay_where_they_are():
    a, d = _inputs(40, 136, "bf16", "channel")
    a["x"][3, 7] = float("inf")
    a["y"][11, 0] = float("nan")
    da, dd = _dev(a), _dev(d)
    got = moe_block_norm(**da, eps=EPS)
    for t in (got.x_out, got.n_out):
        rows = (~torch.isfinite(t)).any(1).nonzero()[:, 0].tolist()
        assert rows == [3, 11]
    g = moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=got.rstd_post,
                                rstd_pre=got.rstd_pre)
    for t in (g.d_x, g.d_y):
        rows = (~torch.isfinite(t)).any(1).nonzero()[:, 0].tolist()
        assert set(rows) <= {3, 11}
    # without the norm ahead of the next block the gradient of x does not see x at all
    g = moe_block_norm_backward(dd["d_x_out"], None, **{**da, "w_pre": None},
                                rstd_post=got.rstd_post)
    assert torch.equal(g.d_x, dd["d_x_out"])


def test_empty_batch_gives_zero_sums():
    a, d = _inputs(0, 136, "bf16", "channel")
    da, dd = _dev(a), _dev(d)
    got = moe_block_norm(**da)
    assert got.x_out.shape == (0, 136) and got.rstd_pre.shape == (0,)
    sums = {k: torch.full((136,), float("nan"), device=DEV) for k in
            ("d_w_post", "d_w_pre", "d_gate")}
    moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=got.rstd_post,
                            rstd_pre=got.rstd_pre, **sums)
    for v in sums.values():
        assert not v.any()


def test_in_place():
    a, d = _inputs(70, 520, "bf16", "token")
    da, dd = _dev(a), _dev(d)
    want = moe_block_norm(**da)
    wg = moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=want.rstd_post,
                                 rstd_pre=want.rstd_pre)
    gx = dd["d_x_out"].clone()
    g = moe_block_norm_backward(gx, dd["d_n_out"], **da, rstd_post=want.rstd_post,
                                rstd_pre=want.rstd_pre, d_x=gx)
    assert g.d_x is gx and torch.equal(gx, wg.d_x) and torch.equal(g.d_y, wg.d_y)
    x = da["x"].clone()
    got = moe_block_norm(**{**da, "x": x}, x_out=x)
    assert got.x_out is x and torch.equal(x, want.x_out) and torch.equal(got.n_out, want.n_out)


def test_same_bits_every_run_and_on_another_stream():
    a, d = _inputs(3001, 264, "bf16", "channel")
    da, dd = _dev(a), _dev(d)

    def run(stream=None):
        f = moe_block_norm(**da, stream=stream)
        g = moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=f.rstd_post,
                                    rstd_pre=f.rstd_pre, stream=stream)
        return [f.x_out, f.n_out, f.rstd_post, f.rstd_pre, g.d_x, g.d_y, g.d_w_post, g.d_w_pre,
                g.d_gate]

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = run(side)
    side.synchronize()
    for u, v in zip(first, second):
        assert torch.equal(u, v)


def test_captured_calls_replay_like_eager_ones():
    a, d = _inputs(130, 264, "bf16", "channel")
    da, dd = _dev(a), _dev(d)
    f = prepare_block_norm(**da)
    out = f.result
    b = prepare_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=out.rstd_post,
                                    rstd_pre=out.rstd_pre)
    grads = b.result
    names = ("d_x", "d_y", "d_w_post", "d_w_pre", "d_gate")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        s = torch.cuda.current_stream()
        moe_block_norm(**da, x_out=out.x_out, n_out=out.n_out, rstd_post=out.rstd_post,
                       rstd_pre=out.rstd_pre, stream=s)
        moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=out.rstd_post,
                                rstd_pre=out.rstd_pre, stream=s,
                                **{k: getattr(grads, k) for k in names})
    for rep in range(4):
        g = torch.Generator().manual_seed(rep)
        for t in (da["x"], da["y"], dd["d_x_out"], dd["d_n_out"]):
            t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        wf = moe_block_norm(**da)
        wg = moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, rstd_post=wf.rstd_post,
                                     rstd_pre=wf.rstd_pre)
        assert torch.equal(out.x_out, wf.x_out) and torch.equal(out.n_out, wf.n_out), rep
        for k in names:
            assert torch.equal(getattr(grads, k), getattr(wg, k)), (rep, k)


def test_gradient_against_differences():
    # central differences of the forward kernel itself, in fp32 with a large step
    a, d = _inputs(4, 64, "f32", "channel", seed=5)
    da, dd = _dev(a), _dev(d)
    f = moe_block_norm(**da, residual_scale=0.5)
    g = moe_block_norm_backward(dd["d_x_out"], dd["d_n_out"], **da, residual_scale=0.5,
                                rstd_post=f.rstd_post, rstd_pre=f.rstd_pre)

    def loss():
        r = moe_block_norm(**da, residual_scale=0.5)
        return float((r.x_out.double() * dd["d_x_out"].double()).sum()
                     + (r.n_out.double() * dd["d_n_out"].double()).sum())

    # rounding of the outputs (|loss terms| sum < 512 * 2^-24 each way) over 2 * step,
    # and step^2 / 6 times a third derivative of order one
    step = 2.0 ** -6
    for name in ("x", "y", "w_post", "w_pre", "gate"):
        t, grad = da[name].view(-1), _np(getattr(g, "d_" + name)).reshape(-1)
        for i in range(0, t.numel(), 37):
            old = float(t[i])
            t[i] = old + step
            up = loss()
            t[i] = old - step
            diff = (up - loss()) / (2 * step)
            t[i] = old
            assert abs(diff - grad[i]) <= 512 * U32 / step + step ** 2, (name, i)


def test_refusals():
    a, d = _inputs(8, 64, "bf16", "token")
    da, dd = _dev(a), _dev(d)

    def fwd(**kw):
        return moe_block_norm(**{**da, **kw})

    def bwd(d_x_out=dd["d_x_out"], d_n_out=dd["d_n_out"], **kw):
        ok = torch.ones(8, device=DEV)
        return moe_block_norm_backward(d_x_out, d_n_out,
                                       **{**da, "rstd_post": ok, "rstd_pre": ok, **kw})

    bf = dict(dtype=torch.bfloat16, device=DEV)
    for call in (fwd, bwd):
        for bad in ({"y": torch.zeros(8, 72, **bf)}, {"w_post": torch.zeros(72, **bf)},
                    {"w_pre": torch.zeros(8, 64, **bf)}, {"gate": torch.zeros(8, 64, **bf)},
                    {"gate": torch.zeros(8, **bf)}, {"y": None}, {"x": a["x"]},
                    {"x": torch.zeros(64, 8, **bf).t()}):
            with pytest.raises(ValueError):
                call(**bad)
        for bad in ({"w_post": torch.zeros(64, device=DEV)}, {"y": da["y"].float()}):
            with pytest.raises(TypeError):
                call(**bad)
    with pytest.raises(ValueError):
        fwd(y=None, w_post=None, gate=None, w_pre=None)
    with pytest.raises(ValueError):
        fwd(w_pre=None, n_out=torch.zeros(8, 64, **bf))
    with pytest.raises(ValueError):
        fwd(x_out=torch.zeros(8, 64, device=DEV))
    for eps in (0.0, -1.0, float("nan")):
        with pytest.raises(MoeError):
            fwd(eps=eps)
    with pytest.raises(MoeError):
        fwd(residual_scale=float("inf"))
    with pytest.raises(MoeError):  # wider than a row may be
        moe_block_norm(torch.zeros(1, 16392, **bf), w_pre=torch.zeros(16392, **bf))
    with pytest.raises(ValueError):
        bwd(d_n_out=None)
    with pytest.raises(ValueError):
        bwd(rstd_post=None)
    with pytest.raises(ValueError):
        bwd(d_gate=torch.zeros(8, device=DEV))
    with pytest.raises(ValueError):
        bwd(d_x_out=None, d_n_out=None, w_pre=None)
    with pytest.raises(MoeError):
        bwd(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
