"""The oracle's gradient of the expert FFN against central differences of its
forward loop, its AdamW step against torch's and its e4m3 values against torch's
float8 type (CPU)."""
import numpy as np
import pytest
import torch

import oracle

STEP = 1e-5

ACTS = [("silu", "packed", {}), ("silu", "interleaved", {"limit": 0.8}),
        ("swiglu_oai", "interleaved", {"alpha": 1.702, "beta": 1.0, "limit": 0.7}),
        ("swiglu_oai", "packed", {"alpha": 1.3, "beta": 0.5}), ("relu2", "packed", {})]


def _differences(f, a):
    """d f / d a by central differences, f scalar."""
    g = np.zeros_like(a)
    flat, out = a.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        old = flat[i]
        flat[i] = old + STEP
        up = f()
        flat[i] = old - STEP
        out[i] = (up - f()) / (2 * STEP)
        flat[i] = old
    return g


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("act,layout,params", ACTS)
def test_ffn_gradient_is_the_derivative(act, layout, params, share):
    rng = np.random.default_rng(3)
    n, e, k, hidden, inter = 5, 4, 2, 3, 4
    idx = np.stack([rng.permutation(e)[:k] for _ in range(n)])
    if share:  # a share of experts 1 and 2
        idx = np.where((idx >= 1) & (idx <= 2), idx - 1, -1)
        e = 2
    order = np.argsort(np.where(idx.reshape(-1) < 0, e, idx.reshape(-1)), kind="stable")
    row = np.empty(n * k, dtype=np.int64)
    row[order] = np.arange(n * k)
    row = row.reshape(n, k)
    rows13 = inter if act == "relu2" else 2 * inter
    x, d = rng.normal(size=(n, hidden)), rng.normal(size=(n, hidden))
    w13, w2 = rng.normal(size=(e, rows13, hidden)), rng.normal(size=(e, hidden, inter))
    w = rng.random((n, k))
    h = np.zeros((n * k, rows13))
    for t in range(n):
        for j in range(k):
            if idx[t, j] >= 0:
                h[row[t, j]] = w13[idx[t, j]] @ x[t]
    got = oracle.moe_ffn_grad(d, x, h, idx, w, row, w13, w2, act, layout, params)

    def total():
        return float((oracle.moe_ffn(x, idx, w, w13, w2, act, layout, params) * d).sum())
    # (no product lies within 100 steps of a kink of the activation)
    lim = params.get("limit", 0.0)
    assert np.abs(np.abs(h[row[idx >= 0]]) - lim).min() > 100 * STEP
    for name, a in (("d_x", x), ("d_w13", w13), ("d_w2", w2), ("d_topk_w", w)):
        want = _differences(total, a)
        # truncation ~ STEP^2 * third derivatives, rounding ~ 2^-53 * |f| / STEP
        assert np.allclose(got[name], want, rtol=1e-6, atol=1e-7), name


def test_activation_gradient_at_the_limit_is_that_of_the_inside():
    g, u = np.array([2.0, 2.0, 3.0]), np.array([2.0, -2.0, 1.0])
    dg, du = oracle.activation_grad("silu", g, u, {"limit": 2.0})
    assert dg[0] != 0 and dg[2] == 0 and du[0] != 0 and du[1] != 0


def test_adamw_is_torchs():
    rng = np.random.default_rng(4)
    hyper = {"lr": 3e-3, "beta1": 0.8, "beta2": 0.97, "eps": 1e-7, "weight_decay": 0.2}
    p = rng.normal(size=50)
    leaf = torch.tensor(p, requires_grad=True)
    opt = torch.optim.AdamW([leaf], lr=hyper["lr"], betas=(hyper["beta1"], hyper["beta2"]),
                            eps=hyper["eps"], weight_decay=hyper["weight_decay"])
    m, v = np.zeros(50), np.zeros(50)
    for step in range(1, 8):
        g = rng.normal(size=50)
        leaf.grad = torch.tensor(g)
        opt.step()
        p, m, v = oracle.adamw(p, g, m, v, step=step, **hyper)
        # float64 on both sides, in another order of operations
        assert np.allclose(p, leaf.detach().numpy(), rtol=1e-13, atol=1e-14)


def test_e4m3_values_are_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(oracle.e4m3_values(), codes.double().numpy())
    assert oracle.e4m3_values()[-1] == 448.0
