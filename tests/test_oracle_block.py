"""The oracle's gradients against central differences of its forward functions,
and its forward functions against closed forms (CPU)."""
import numpy as np
import pytest

import oracle

STEP = 1e-5


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


def _close(got, want):
    # truncation ~ STEP^2 * third derivatives, rounding ~ 2^-53 * |f| / STEP
    assert np.allclose(got, want, rtol=1e-6, atol=1e-7), np.abs(got - want).max()


def _sorted_order(rng, n, e, k):
    idx = np.stack([rng.permutation(e)[:k] for _ in range(n)])
    col = np.argsort(idx.reshape(-1), kind="stable")
    row = np.empty_like(col)
    row[col] = np.arange(n * k)
    return idx, row


def test_dispatch_and_combine_are_inverse_for_weights_that_sum_to_one():
    rng = np.random.default_rng(0)
    n, e, k, h = 7, 5, 3, 4
    _, row = _sorted_order(rng, n, e, k)
    x = rng.normal(size=(n, h))
    w = rng.random((n, k))
    w /= w.sum(1, keepdims=True)
    xs = oracle.dispatch(x, row, k)
    assert np.array_equal(xs[row], np.repeat(x, k, axis=0))
    _close(oracle.combine_weighted(xs, row, w), x)


@pytest.mark.parametrize("share", [False, True])
def test_combine_gradient_is_the_derivative(share):
    rng = np.random.default_rng(1)
    n, e, k, h = 5, 4, 2, 3
    idx, row = _sorted_order(rng, n, e, k)
    if share:  # experts 0 and 1 only: the other slots are skipped
        local = idx.reshape(-1) < 2
        rank = np.argsort(np.argsort(np.where(local, idx.reshape(-1) * 100, 10 ** 6),
                                     kind="stable"), kind="stable")
        row = np.where(local, rank, -1)
    y, d = rng.normal(size=(n * k, h)), rng.normal(size=(n, h))
    logits = rng.normal(size=(n, e))

    def weights():
        v = np.take_along_axis(logits, idx, 1)
        p = np.exp(v - v.max(1, keepdims=True))
        return p / p.sum(1, keepdims=True)

    def loss():
        return float((oracle.combine_weighted(y, row, weights()) * d).sum())

    dy, dw = oracle.combine_weighted_grad(d, y, row, weights())
    _close(dy, _differences(loss, y))
    _close(oracle.topk_weight_grad(dw, idx, weights(), e), _differences(loss, logits))


@pytest.mark.parametrize("gate,branch,post,pre", [
    (g, 1, post, pre) for g in ("none", "token", "channel") for post in (0, 1) for pre in (0, 1)
] + [("none", 0, 0, 1)])
def test_block_norm_gradient_is_the_derivative(gate, branch, post, pre):
    rng = np.random.default_rng(2)
    n, h = 3, 5
    a = {"x": rng.normal(size=(n, h)), "y": rng.normal(size=(n, h)) if branch else None,
         "w_post": rng.normal(size=h) if post else None,
         "w_pre": rng.normal(size=h) if pre else None,
         "gate": {"none": None, "token": rng.normal(size=(n, 1)),
                  "channel": rng.normal(size=h)}[gate]}
    d_x, d_n = rng.normal(size=(n, h)), rng.normal(size=(n, h)) if pre else None

    def loss():
        f = oracle.block_norm(**a, scale=0.3, eps=1e-3)
        x_out = a["x"] if f["x_out"] is None else f["x_out"]
        return float((x_out * d_x).sum() + ((f["n_out"] * d_n).sum() if pre else 0.0))

    g = oracle.block_norm_grad(d_x, d_n, **a, scale=0.3, eps=1e-3)
    for name, v in a.items():
        if v is None:
            assert g["d_" + name] is None
        else:
            _close(g["d_" + name], _differences(loss, v))


def test_rms_norm_closed_forms():
    u = np.array([[3.0, -3.0, 3.0, -3.0], [0.0, 0.0, 0.0, 0.0]])
    n, r = oracle.rms_norm(u, np.array([1.0, 1.0, 2.0, 0.5]), 0.25)
    assert np.allclose(r, [1 / np.sqrt(9.25), 2.0])  # an all-zero row: 1 / sqrt(eps)
    assert np.allclose(n[0], np.array([3, -3, 6, -1.5]) / np.sqrt(9.25))
    assert not n[1].any()
