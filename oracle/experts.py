"""The MoE gate, the experts' products and their gradients in binary64
(oracle; test infrastructure only).

The pages describe no expert computation (the SiFAR review only evaluates a
large MoE model end to end); these are the usual definitions, on numpy float64
arrays:

* gate: p = softmax(l) over the scores that are not -inf; the top-k by
  descending score, ties to the lower expert; w = p of the chosen ones, or
  p / (their sum);
* linear: Y = act(X W^T + b) + R, per group of rows;
* gated: H = act(X Wg^T) * (X Wu^T), per group of rows.

Pinned by central differences of every gradient and by hand-made cases
(tests/test_oracle_experts.py).
"""

import numpy as np
from scipy.special import erfc

ACTIVATIONS = ("none", "silu", "gelu", "gelu_tanh", "relu")
_C = np.sqrt(2.0 / np.pi)


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def act(name, x):
    if name == "silu":
        return x * _sigmoid(x)
    if name == "gelu":
        return 0.5 * x * erfc(-x / np.sqrt(2.0))
    if name == "gelu_tanh":
        return x * _sigmoid(2.0 * _C * (x + 0.044715 * x ** 3))
    if name == "relu":
        return np.maximum(x, 0.0)
    return x


def act_grad(name, x):
    if name == "silu":
        s = _sigmoid(x)
        return s * (1.0 + x * (1.0 - s))
    if name == "gelu":
        return 0.5 * erfc(-x / np.sqrt(2.0)) + x * np.exp(-0.5 * x * x) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        s = _sigmoid(2.0 * _C * (x + 0.044715 * x ** 3))
        return s + x * s * (1.0 - s) * 2.0 * _C * (1.0 + 3 * 0.044715 * x * x)
    if name == "relu":
        return (x > 0).astype(np.float64)
    return np.ones_like(x)


def groups(offsets):
    """(group, rows as a slice) of every group that has rows."""
    return [(e, slice(int(a), int(b))) for e, (a, b) in enumerate(zip(offsets, offsets[1:])) if b > a]


def linear(x, offsets, w, bias=None, name="none", residual=None):
    """(Y, pre-activation); rows outside the groups are NaN."""
    pre = np.full((x.shape[0], w.shape[1]), np.nan)
    for e, r in groups(offsets):
        pre[r] = x[r] @ w[e].T + (0.0 if bias is None else bias[e])
    y = act(name, pre)
    return (y if residual is None else y + residual), pre


def linear_grad(d_y, x, offsets, w, pre=None, name="none"):
    """(dX, dW, db) at the given pre-activation values."""
    d = d_y if name == "none" else d_y * act_grad(name, pre)
    d_x, d_w = np.full(x.shape, np.nan), np.zeros(w.shape)
    d_b = np.zeros(w.shape[:2])
    for e, r in groups(offsets):
        d_x[r] = d[r] @ w[e]
        d_w[e] = d[r].T @ x[r]
        d_b[e] = d[r].sum(axis=0)
    return d_x, d_w, d_b


def gated(x, offsets, w_gate, w_up, name):
    """(H, gate, up); rows outside the groups are NaN."""
    _, g = linear(x, offsets, w_gate)
    _, u = linear(x, offsets, w_up)
    return act(name, g) * u, g, u


def gated_grad(d_h, x, offsets, w_gate, w_up, g, u, name):
    """(dX, dWg, dWu) at the given projections."""
    xg, wg, _ = linear_grad(d_h * u * act_grad(name, g), x, offsets, w_gate)
    xu, wu, _ = linear_grad(d_h * act(name, g), x, offsets, w_up)
    return xg + xu, wg, wu


def gate(logits, k, renormalize=False):
    """(idx [T, k], w [T, k]) of float64 scores without NaN or +inf."""
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(softmax(logits), idx, axis=1)
    if renormalize:
        s = w.sum(axis=1, keepdims=True)
        w = w / np.where(s == 0, 1.0, s)
    return idx, w


def softmax(logits):
    m = logits.max(axis=1, keepdims=True)
    e = np.where(np.isneginf(logits), 0.0, np.exp(logits - np.where(np.isneginf(m), 0.0, m)))
    s = e.sum(axis=1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def gate_grad(logits, idx, d_w, renormalize=False):
    p = softmax(logits)
    live = ~np.isneginf(np.take_along_axis(logits, idx, axis=1))
    d = np.where(live, d_w, 0.0)
    full, on = np.zeros_like(p), np.zeros_like(p)
    np.put_along_axis(full, idx, d, axis=1)
    np.put_along_axis(on, idx, live.astype(np.float64), axis=1)
    if renormalize:
        s = (p * on).sum(axis=1, keepdims=True)
        w = p * on / np.where(s == 0, 1.0, s)
        return w * (full - (w * full).sum(axis=1, keepdims=True))
    return p * (full - (p * full).sum(axis=1, keepdims=True))


def combine_grad(d_y, z, slot, w):
    """(dz, dw) of y[t] = sum over j of w[t, j] z[slot[t, j]]."""
    d_z = np.zeros_like(z)
    d_z[slot.reshape(-1)] = (w[:, :, None] * d_y[:, None, :]).reshape(-1, z.shape[1])
    return d_z, (d_y[:, None, :] * z[slot]).sum(axis=2)
