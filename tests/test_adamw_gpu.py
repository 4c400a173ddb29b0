"""AdamW over many tensors and the gradient norm on the GPU against the float64
oracle.

Tolerances (U = 2^-24, half a step of fp32).  g = grad coef, m and v are three to
five roundings of their terms: 6 U of the terms' magnitudes.  The update is a product
of a constant, m, and the hardware's reciprocal (a step) of a root: 24 U of c1 |m'| /
(c2 root + eps) with m' the terms' magnitudes; p adds 4 U of its own terms and half a
step of its type.  An 8-bit value is one of its two e4m3 neighbours (stochastic) or
the nearest (up to the same fp32 errors at the border)."""
import numpy as np
import pytest
import torch

import oracle
from routing_grouped_expert_amd import (AdamWState, MoeError, moe_adamw, moe_adamw_state,
                                        moe_grad_norm, prepare_adamw, prepare_grad_norm)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HYPER = {"lr": 2e-3, "betas": (0.9, 0.99), "eps": 1e-8, "weight_decay": 0.1}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def _within(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst " \
                          f"{np.nanmax(err / np.maximum(tol, 1e-300)):.3g} tolerances, first at " \
                          f"{int(np.argwhere(bad)[0][0])}"


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _problem(sizes, p_dtype, g_dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    params = [(torch.randn(s, generator=g) * 0.05).to(DT[p_dtype]) for s in sizes]
    grads = [(torch.randn(s, generator=g) * 1e-2 *
              (1 + 30 * (torch.rand(s, generator=g) < 0.01))).to(DT[g_dtype]) for s in sizes]
    return params, grads


def _moments(state, i):
    """(m, v) of tensor i as float64 arrays."""
    if state.m_scale is None:
        return _np(state.m[i]), _np(state.v[i])
    n = state.m[i].numel()
    m = _np(state.m[i].float()) * np.repeat(_np(state.m_scale[i]), 256)[:n]
    r = _np(state.v[i].float()) * np.repeat(_np(state.v_scale[i]), 256)[:n]
    return m, r * r


def _neighbours(x, scale, stochastic):
    """Smallest and largest value that x (float64) may be held as."""
    vals = np.concatenate([-oracle.e4m3_values()[:0:-1], oracle.e4m3_values()])
    s = np.repeat(scale, 256)[:len(x)]
    u = np.divide(x, s, out=np.zeros_like(x), where=s > 0)
    slack = 64 * U * np.abs(u)
    lo, hi = np.clip(u - slack, -448, 448), np.clip(u + slack, -448, 448)
    if stochastic:
        below = vals[np.clip(np.searchsorted(vals, lo, side="right") - 1, 0, len(vals) - 1)]
        above = vals[np.clip(np.searchsorted(vals, hi, side="left"), 0, len(vals) - 1)]
    else:
        mid = (vals[1:] + vals[:-1]) / 2
        below = vals[np.searchsorted(mid, lo, side="left")]
        above = vals[np.searchsorted(mid, hi, side="right")]
    return below * s, above * s


def _check_step(params, grads, state, step, coef, seed, run, hyper=HYPER):
    """One step on the GPU (``run``) against the oracle's from the same values."""
    before = [(_np(p), *_moments(state, i),
               _np(state.master[i]) if state.master and state.master[i] is not None else None)
              for i, p in enumerate(params)]
    run()
    b1, b2 = hyper["betas"]
    for i, (p0, m0, v0, w0) in enumerate(before):
        if p0.size == 0:
            continue
        p, base = params[i], p0 if w0 is None else w0
        g = _np(grads[i])
        args = {"lr": hyper["lr"], "beta1": b1, "beta2": b2, "eps": hyper["eps"],
                "weight_decay": hyper["weight_decay"], "step": step, "coef": coef}
        w, m, v = oracle.adamw(base, g, m0, v0, **args)
        mt = b1 * np.abs(m0) + (1 - b1) * np.abs(g) * coef
        c1, c2 = hyper["lr"] / (1 - b1 ** step), 1 / (1 - b2 ** step) ** 0.5
        tol_w = 24 * U * c1 * mt / (c2 * np.sqrt(v) + hyper["eps"]) + 4 * U * np.abs(base) + 1e-37
        if w0 is not None:
            got = _np(state.master[i])
            _within(got, w, tol_w + U * np.abs(w), f"master {i}")
            assert torch.equal(params[i], state.master[i].to(p.dtype)), f"p {i} is not its master's"
        elif seed is not None and p.dtype == torch.bfloat16:
            # one of the two neighbours: less than a whole step (of the binade above)
            _within(_np(p), w, tol_w + 2 * _half(p.dtype) * np.abs(w) * (1 + 1e-3) + 1e-37, f"p {i}")
        else:
            _within(_np(p), w, tol_w + _half(p.dtype) * np.abs(w), f"p {i}")
        if state.m_scale is None:
            _within(_np(state.m[i]), m, 6 * U * mt + 1e-37, f"m {i}")
            _within(_np(state.v[i]), v, 6 * U * v + 1e-37, f"v {i}")
            continue
        root = np.sqrt(v)
        for name, x, q, scale in (("m", m, state.m[i], state.m_scale[i]),
                                  ("r", root, state.v[i], state.v_scale[i])):
            sc, want = _np(scale), oracle.block_scale(x)
            _within(sc, want, 16 * U * want * (1 + mt.max() / max(np.abs(m).max(), 1e-300)) + 1e-44,
                    f"{name}_scale {i}")
            got = _np(q.float()) * np.repeat(sc, 256)[:x.size]
            lo, hi = _neighbours(x, sc, seed is not None)
            cancel = 16 * U * mt if name == "m" else 16 * U * root  # m's terms may cancel
            if name == "r":  # nothing above zero becomes zero
                least = np.repeat(sc, 256)[:x.size] * 2.0 ** -9
                live = (x > 1e-30) & (least > 0)
                assert (got[live] > 0).all()
                hi = np.maximum(hi, least)
            bad = (got < lo - cancel) | (got > hi + cancel)
            assert not bad.any(), f"{name} {i}: {int(bad.sum())} values are no neighbours, first " \
                                  f"{int(np.argwhere(bad)[0][0])}"


SIZES = [(1,), (7,), (8,), (0,), (255,), (256,), (257,), (3, 5, 7), (2048,), (8192,), (8193,),
         (30000,), (64, 1001)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                 ("f32", "bf16")])
@pytest.mark.parametrize("master,seed", [(False, None), (False, 7), (True, 7), (True, None)])
def test_steps(bits, p, g, master, seed):
    params, grads = _problem(SIZES, p, g)
    params = [t.to(DEV) for t in params]
    state = moe_adamw_state(params, bits, master=master)
    for step in (1, 2, 3):
        _, grads = _problem(SIZES, p, g, seed=step)
        grads = [t.to(DEV) for t in grads]
        norm = moe_grad_norm(grads)
        exact = np.sqrt(sum(float((_np(t) ** 2).sum()) for t in grads))
        # each square is rounded to fp32 once, the sum and the root are in 64 bits
        assert norm.dtype == torch.float64 and abs(float(norm) - exact) <= U * exact
        clip = 0.5 * exact if step == 2 else None
        coef = 1.0 if clip is None else oracle.clip_coefficient(float(norm), clip)
        _check_step(params, grads, state, step, coef, seed, lambda: moe_adamw(
            params, grads, state, step=step, seed=seed, grad_norm=None if clip is None else norm,
            max_norm=clip, **HYPER))


def test_more_tensors_than_a_launch_takes():
    sizes = [(i % 9 * 37,) for i in range(101)]
    params, grads = _problem(sizes, "f32", "f32")
    params, grads = [t.to(DEV) for t in params], [t.to(DEV) for t in grads]
    state = moe_adamw_state(params, 8)
    exact = np.sqrt(sum(float((_np(t) ** 2).sum()) for t in grads))
    assert abs(float(moe_grad_norm(grads)) - exact) <= U * exact
    _check_step(params, grads, state, 1, 1.0, 5, lambda: moe_adamw(
        params, grads, state, step=1, seed=5, **HYPER))
    # the same bits every time, and others with another seed, step or place
    again = [[t.clone() for t in ts] for ts in (params, state.m, state.v)]
    first = None
    for seed, step in ((5, 2), (5, 2), (6, 2), (5, 3)):
        ps, ms, vs = [[t.clone() for t in ts] for ts in again]
        st = AdamWState(ms, vs, [t.clone() for t in state.m_scale],
                        [t.clone() for t in state.v_scale])
        moe_adamw(ps, grads, st, step=step, seed=seed, **HYPER)
        got = torch.cat([t.view(torch.uint8) for t in ms if t.numel()])
        if first is None:
            first = got
        else:
            assert torch.equal(first, got) == ((seed, step) == (5, 2))


def test_stochastic_rounding_has_the_mean_of_what_it_rounds():
    """A bf16 weight between two values: over 2^16 elements the mean is off by less
    than five standard deviations of the rounding (a step / 2 / 2^8), and by 2^-12 of a
    step that 12 random bits may leave."""
    n, value = 1 << 16, 1.0 + 2.0 ** -7 * 0.3  # a third of the way up
    p = torch.ones(n, device=DEV, dtype=torch.bfloat16)
    g = torch.zeros(n, device=DEV)
    state = moe_adamw_state([p], 32)
    # decay alone moves the weight: p (1 - lr wd) = value
    moe_adamw([p], [g], state, step=1, lr=1.0, weight_decay=0.0, seed=3)
    assert torch.equal(p, torch.ones_like(p))  # exact values stay
    state = moe_adamw_state([p], 32)
    q = torch.full((n,), 2.0, device=DEV, dtype=torch.bfloat16)
    moe_adamw([q], [g], state, step=1, lr=1.0, weight_decay=1.0 - value / 2, seed=3)
    step = 2.0 ** -7
    assert set(q.unique().tolist()) == {1.0, 1.0 + step}
    assert abs(float(q.double().mean()) - value) <= step * (5 / 2 / 2 ** 8 + 2.0 ** -11)


def test_small_second_moments_stay_above_zero_and_zeros_stay_zero():
    n = 512
    g = torch.full((n,), 1e-6, device=DEV)
    g[0], g[300:] = 1e3, 0.0
    p = torch.zeros(n, device=DEV)
    state = moe_adamw_state([p], 8)
    moe_adamw([p], [g], state, step=1, lr=1e-3, weight_decay=0.0, eps=1e-12)
    r = state.v[0].float()
    assert (r[:256] > 0).all() and (r[300:] == 0).all() and (p[300:] == 0).all()
    assert float(p.abs().max()) <= 1e-3 * (1 + 1e-5)  # (no step beyond lr)
    # a block of zeros holds zeros
    zero = torch.zeros(n, device=DEV)
    state = moe_adamw_state([p], 8)
    before = p.clone()
    moe_adamw([p], [zero], state, step=1, lr=1e-3, weight_decay=0.0)
    assert torch.equal(p, before) and not state.m_scale[0].any() and not state.v_scale[0].any()


def test_a_norm_that_is_not_finite_skips_the_step_and_without_one_nan_shows():
    for bad in (float("inf"), float("nan")):
        g = torch.ones(1000, device=DEV)
        g[700] = bad
        p = torch.ones(1000, device=DEV)
        state = moe_adamw_state([p], 8)
        norm = moe_grad_norm([g])
        assert not torch.isfinite(norm).any()
        moe_adamw([p], [g], state, step=1, lr=0.1, grad_norm=norm, max_norm=1.0)
        assert torch.equal(p, torch.ones_like(p)) and not state.m[0].float().any()
        moe_adamw([p], [g], state, step=1, lr=0.1)
        scale = state.v_scale[0]
        assert torch.isnan(scale[2]) and torch.isfinite(scale[[0, 1, 3]]).all()
        assert not torch.isfinite(p[700]) and torch.isfinite(p[:700]).all()


def test_capture_counts_the_step_on_the_device():
    sizes = [(300,), (5000,)]
    params, grads = _problem(sizes, "bf16", "f32")
    grads = [t.to(DEV) for t in grads]
    eager = [t.to(DEV) for t in params]
    graphed = [t.clone() for t in eager]
    se, sg = moe_adamw_state(eager, 8), moe_adamw_state(graphed, 8)
    step = torch.zeros(1, dtype=torch.int32, device=DEV)
    norm = torch.empty(1, dtype=torch.float64, device=DEV)
    call_norm = prepare_grad_norm(grads, out=norm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step.add_(1)
        moe_grad_norm(grads, out=norm, stream=side)
        moe_adamw(graphed, grads, sg, step=step, grad_norm=norm, max_norm=0.1, seed=9, **HYPER)
    assert int(step) == 0
    for t in (1, 2, 3, 4):
        graph.replay()
        torch.cuda.synchronize()
        call_norm()
        prepare_adamw(eager, grads, se, step=torch.tensor([t], dtype=torch.int32, device=DEV),
                      grad_norm=norm, max_norm=0.1, seed=9, **HYPER)()
        torch.cuda.synchronize()
        assert int(step) == t
        for a, b in zip(eager + se.m_scale + se.v_scale, graphed + sg.m_scale + sg.v_scale):
            assert torch.equal(a, b)
        for a, b in zip(se.m + se.v, sg.m + sg.v):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_another_stream():
    params, grads = _problem([(70001,)], "f32", "f32")
    p, g = params[0].to(DEV), grads[0].to(DEV)
    state = moe_adamw_state([p], 32)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())

    def run():
        norm = moe_grad_norm([g], stream=other)
        moe_adamw([p], [g], state, step=1, grad_norm=norm, max_norm=1e9, stream=other, **HYPER)
        other.synchronize()
    _check_step([p], [g], state, 1, 1.0, None, run)


def test_refusals():
    p, g = torch.ones(16, device=DEV), torch.ones(16, device=DEV)
    s = moe_adamw_state([p])
    ok = {"lr": 1e-3, "step": 1}
    with pytest.raises(ValueError):
        moe_adamw([p, p], [g, g.clone()], moe_adamw_state([p, p]), **ok)      # twice the same
    with pytest.raises(ValueError):
        moe_adamw([p], [p], s, **ok)                                          # p is its gradient
    both = torch.ones(32, device=DEV)
    with pytest.raises(ValueError):
        moe_adamw([both[:20], both[16:]], [g[:4].repeat(5), g], moe_adamw_state(
            [both[:20], both[16:]]), **ok)                                    # they overlap
    for bad in ([g[:8]], [g.half()], [g.cpu()], [torch.ones(32, device=DEV)[::2]], []):
        with pytest.raises((ValueError, TypeError)):
            moe_adamw([p], bad, s, **ok)
    with pytest.raises(ValueError):
        moe_adamw([p], [g], moe_adamw_state([p, p]), **ok)
    with pytest.raises(ValueError):
        moe_adamw([p], [g], AdamWState(s.m, [t.half() for t in s.v]), **ok)
    with pytest.raises(ValueError):
        moe_adamw([p], [g], s, grad_norm=torch.ones(1, device=DEV, dtype=torch.float64), **ok)
    with pytest.raises((ValueError, TypeError)):  # not in 64 bits
        moe_adamw([p], [g], s, grad_norm=torch.ones(1, device=DEV), max_norm=1.0, **ok)
    for bad in ({"step": 0}, {"step": 1 << 31}, {"lr": -1.0}, {"lr": float("nan")},
                {"betas": (1.0, 0.9)}, {"betas": (0.9, -0.1)}, {"eps": float("inf")},
                {"weight_decay": -0.1}):
        with pytest.raises(MoeError):
            moe_adamw([p], [g], s, **{**ok, **bad})
    with pytest.raises(MoeError):  # 16-byte alignment
        q = torch.ones(17, device=DEV)[1:]
        moe_adamw([q], [g], s, **ok)
    with pytest.raises(ValueError):
        moe_grad_norm([])
    assert torch.equal(p, torch.ones_like(p))
