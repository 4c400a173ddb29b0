"""Oracle of the steps around the experts (test infrastructure only; see the
package docstring): rows into expert-sorted order and back with the routing
weights, the norms around a block, and their gradients, in float64.

* ``dispatch`` / ``combine_weighted`` are the sort-by-expert dispatch and the
  weighted sum back of the minimind issue #835 page ("It is removable in plain
  PyTorch"), as loops over the entries; slots whose position is negative
  (outside an expert share) are skipped.
* ``block_norm`` is ``x + s * gate * rmsnorm(y)`` followed by the next norm.
* The ``*_grad`` functions are the derivatives, pinned by central differences
  of the forward functions in ``tests/test_oracle_block.py``.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    if a is None:
        return None
    if not isinstance(a, np.ndarray):  # a torch tensor (bf16 has no numpy type)
        a = a.detach().double().cpu().numpy()
    return a.astype(np.float64)


def dispatch(x, row_sorted, k: int, into=None) -> np.ndarray:
    x, row_sorted = _f64(x), np.asarray(row_sorted).reshape(-1)
    out = np.zeros((len(row_sorted), x.shape[1])) if into is None else _f64(into).copy()
    for f, p in enumerate(row_sorted):
        if p >= 0:
            out[p] = x[f // k]
    return out


def combine_weighted(y, row_sorted, w) -> np.ndarray:
    y, w = _f64(y), _f64(w)
    n, k = w.shape
    out = np.zeros((n, y.shape[1]))
    for t in range(n):
        for j in range(k):
            p = row_sorted[t * k + j]
            if p >= 0:
                out[t] += w[t, j] * y[p]
    return out


def combine_weighted_grad(d_out, y, row_sorted, w, into=None):
    """``(d_y, d_w)``; rows of d_y that no slot points to keep ``into`` (zeros)."""
    d_out, y, w = _f64(d_out), _f64(y), _f64(w)
    n, k = w.shape
    dy = np.zeros_like(y) if into is None else _f64(into).copy()
    dw = np.zeros((n, k))
    for t in range(n):
        for j in range(k):
            p = row_sorted[t * k + j]
            if p >= 0:
                dy[p] = w[t, j] * d_out[t]
                dw[t, j] = d_out[t] @ y[p]
    return dy, dw


def topk_weight_grad(dw, topk_idx, w, n_experts: int) -> np.ndarray:
    """Gradient of the softmax over the selected logits, scattered to [N, E]."""
    dw, w, topk_idx = _f64(dw), _f64(w), np.asarray(topk_idx)
    out = np.zeros((len(w), n_experts))
    for t in range(len(w)):
        inner = float(w[t] @ dw[t])
        for j, e in enumerate(topk_idx[t]):
            out[t, e] = w[t, j] * (dw[t, j] - inner)
    return out


def rms_norm(u, w, eps: float):
    """``(u * rstd * w, rstd)`` with rstd = 1 / sqrt(mean(u^2) + eps) per row."""
    r = 1.0 / np.sqrt((u * u).mean(axis=1) + eps)
    return u * r[:, None] * w, r


def block_norm(x, y=None, w_post=None, w_pre=None, gate=None, scale=1.0, eps=1e-6):
    """Dict of x_out, n_out, rstd_post, rstd_pre (None for what is absent)."""
    x, y, w_post, w_pre, gate = map(_f64, (x, y, w_post, w_pre, gate))
    res = {"x_out": None, "n_out": None, "rstd_post": None, "rstd_pre": None}
    if y is not None:
        z = y
        if w_post is not None:
            z, res["rstd_post"] = rms_norm(y, w_post, eps)
        x = x + scale * (z if gate is None else gate * z)
        res["x_out"] = x
    if w_pre is not None:
        res["n_out"], res["rstd_pre"] = rms_norm(x, w_pre, eps)
    return res


def _rms_grad(u, r, w, d):
    uh = u * r[:, None]
    g = d * w
    return r[:, None] * (g - uh * (g * uh).mean(axis=1, keepdims=True)), (d * uh).sum(axis=0)


def block_norm_grad(d_x_out, d_n_out, x, y=None, w_post=None, w_pre=None, gate=None, scale=1.0,
                    eps=1e-6):
    """Dict of d_x, d_y, d_w_post, d_w_pre, d_gate (None for what is absent)."""
    d_x_out, d_n_out, x, y, w_post, w_pre, gate = map(
        _f64, (d_x_out, d_n_out, x, y, w_post, w_pre, gate))
    f = block_norm(x, y, w_post, w_pre, gate, scale, eps)
    res = {"d_x": None, "d_y": None, "d_w_post": None, "d_w_pre": None, "d_gate": None}
    d = np.zeros_like(x) if d_x_out is None else d_x_out
    if w_pre is not None:
        u = x if y is None else f["x_out"]
        du, res["d_w_pre"] = _rms_grad(u, f["rstd_pre"], w_pre, d_n_out)
        d = d + du
    res["d_x"] = d
    if y is not None:
        z = y if w_post is None else y * f["rstd_post"][:, None] * w_post
        dz = scale * d
        if gate is not None:
            dg = dz * z
            res["d_gate"] = dg.sum(axis=1, keepdims=True) if gate.ndim == 2 else dg.sum(axis=0)
            dz = dz * gate
        if w_post is not None:
            dz, res["d_w_post"] = _rms_grad(y, f["rstd_post"], w_post, dz)
        res["d_y"] = dz
    return res
