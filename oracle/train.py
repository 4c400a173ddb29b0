"""Oracle of a training step of the experts (test infrastructure only; see the
package docstring): the gradient of the expert FFN and the AdamW step, in
float64.

* ``moe_ffn_grad`` differentiates the masked per-expert loop of
  :func:`oracle.ffn.moe_ffn` by hand, with the w13 products ``h`` given (a
  training step saves them rounded); pinned by central differences of that loop
  in ``tests/test_oracle_train.py``.
* ``adamw`` is the decoupled-weight-decay Adam step with bias correction;
  ``e4m3_values`` and ``block_scale`` say what 8-bit moments can hold.  Pinned by
  torch's optimizer and torch's float8 type.
"""
from __future__ import annotations

import numpy as np

from .ffn import activation, split_gate_up

BLOCK, TOP = 256, 448.0


def activation_grad(act: str, g, u=None, params: dict | None = None):
    """Derivatives of :func:`oracle.ffn.activation` with respect to ``g`` and ``u``
    (None for relu2); 0 where a clamp holds, that of the inside at the limit."""
    params = params or {}
    if act == "relu2":
        return 2.0 * np.maximum(g, 0.0), None
    lim = params.get("limit", np.inf)
    alpha, beta = (params.get("alpha", 1.0), params.get("beta", 0.0)) if act == "swiglu_oai" \
        else (1.0, 0.0)
    gc, uc = np.minimum(g, lim), np.clip(u, -lim, lim)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-alpha * gc))
    dg = np.where(g <= lim, (s + alpha * gc * s * (1.0 - s)) * (uc + beta), 0.0)
    return dg, np.where(np.abs(u) <= lim, gc * s, 0.0)


def join_gate_up(g, u, layout: str) -> np.ndarray:
    """Rows in w13 order from their gate and up parts."""
    if layout == "packed":
        return np.concatenate([g, u], axis=-1)
    return np.stack([g, u], axis=-1).reshape(*g.shape[:-1], 2 * g.shape[-1])


def moe_ffn_grad(d_out, x, h, idx, w, row, w13, w2, act: str, layout: str = "packed",
                 params: dict | None = None) -> dict:
    """Gradients of ``sum(out * d_out)`` (all arrays float64): ``idx [N, k]`` local
    expert ids (-1: outside the share), ``w [N, k]`` routing weights, ``row [N, k]``
    the sorted row of each slot, whose w13 products are ``h[row]``."""
    d_w13, d_w2, d_x = np.zeros_like(w13), np.zeros_like(w2), np.zeros_like(x)
    d_w = np.zeros(np.shape(w))
    for e in range(len(w13)):
        tok, slot = np.nonzero(np.asarray(idx) == e)
        he, we, d = h[row[tok, slot]], w[tok, slot][:, None], d_out[tok]
        if act == "relu2":
            a, (dg, _) = activation(act, he), activation_grad(act, he)
        else:
            g, u = split_gate_up(he, layout)
            a, (dg, du) = activation(act, g, u, params), activation_grad(act, g, u, params)
        da = d @ w2[e]
        d_w[tok, slot] = (da * a).sum(axis=1)
        dh = we * da * dg if act == "relu2" else join_gate_up(we * da * dg, we * da * du, layout)
        np.add.at(d_x, tok, dh @ w13[e])
        d_w13[e] = dh.T @ x[tok]
        d_w2[e] = d.T @ (we * a)
    return {"d_x": d_x, "d_w13": d_w13, "d_w2": d_w2, "d_topk_w": d_w}


def adamw(p, grad, m, v, *, lr, beta1, beta2, eps, weight_decay, step, coef=1.0):
    """One step, all arrays float64: ``(p, m, v)`` after it."""
    g = grad * coef
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    update = (m / (1.0 - beta1 ** step)) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps)
    return p - lr * weight_decay * p - lr * update, m, v


def clip_coefficient(norm: float, max_norm: float) -> float:
    return min(1.0, max_norm / (norm + 1e-6))


def e4m3_values() -> np.ndarray:
    """The values of the codes 0 .. 126 of the OCP e4m3 format (sign bit clear; 127 is
    NaN): 4 exponent bits with bias 7, 3 mantissa bits, subnormals below 2^-6."""
    code = np.arange(127)
    ex, man = code >> 3, code & 7
    return np.where(ex == 0, man / 8.0 * 2.0 ** -6, (1 + man / 8.0) * 2.0 ** (ex - 7.0))


def block_scale(x: np.ndarray) -> np.ndarray:
    """Scale of each block of 256 elements of the flat array x."""
    top = np.abs(np.concatenate([x, np.zeros(-len(x) % BLOCK)])).reshape(-1, BLOCK).max(1)
    return np.where(top >= 2.0 ** -100, top / TOP, 0.0)
