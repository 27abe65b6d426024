"""Plain FP64 statement of the training-step operators (include/qlora_train.h), formula by
formula, for the tests only.  It shares nothing with the HIP library; its gradients are pinned
by finite differences of its forwards in ``tests/test_training_oracle.py``."""

from __future__ import annotations

import numpy as np

F = np.float64


def gate_of_rows(gate, gate_rows, M):
    """The gate row of each of M rows (ones without a gate)."""
    return None if gate is None else gate.astype(F)[np.arange(M) // gate_rows]


def _inv_rms(v, eps):
    with np.errstate(divide="ignore"):
        return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def norm_residual_fwd(x, y=None, post_norm=False, w_post=None, gate=None, gate_rows=0, w_pre=None, res_scale=1.0,
                      eps=1e-5):
    """(x', h) of the boundary between two blocks."""
    x = x.astype(F)
    xo = res_scale * x
    if y is not None:
        n = y.astype(F)
        if post_norm:
            n = n * _inv_rms(n, eps)
            if w_post is not None:
                n = n * w_post.astype(F)
        g = gate_of_rows(gate, gate_rows, x.shape[0])
        xo = xo + (n if g is None else g * n)
    h = xo * _inv_rms(xo, eps)
    return xo, h if w_pre is None else h * w_pre.astype(F)


def norm_residual_bwd(xo, y, dh, dxo, post_norm=False, w_post=None, gate=None, gate_rows=0, w_pre=None, res_scale=1.0,
                      eps=1e-5):
    """dict(dx, dy, dw_post, dgate, dw_pre), and the magnitudes that the terms of each sum up to
    ("abs"), for error bounds."""
    first = xo if xo is not None else dxo
    M, d = first.shape
    t = np.zeros((M, d)) if dxo is None else dxo.astype(F)
    t_abs = np.abs(t)
    out, mag = {}, {}
    if dh is not None:
        x, dh = xo.astype(F), dh.astype(F)
        r = _inv_rms(x, eps)
        a = dh if w_pre is None else dh * w_pre.astype(F)
        t = t + r * a - x * r**3 * np.mean(a * x, axis=1, keepdims=True)
        t_abs = t_abs + r * np.abs(a) + np.abs(x) * r**3 * np.mean(np.abs(a * x), axis=1, keepdims=True)
        out["dw_pre"], mag["dw_pre"] = np.sum(dh * x * r, axis=0), np.sum(np.abs(dh * x * r), axis=0)
    out["dx"], mag["dx"] = res_scale * t, np.abs(res_scale) * t_abs
    if y is None:
        return out, mag
    y = y.astype(F)
    g = gate_of_rows(gate, gate_rows, M)
    r = _inv_rms(y, eps) if post_norm else np.ones((M, 1))
    w = w_post.astype(F) if w_post is not None else np.ones(d)
    n = y * r * w
    if g is not None:
        owner = np.arange(M) // gate_rows
        out["dgate"], mag["dgate"] = np.zeros(gate.shape), np.zeros(gate.shape)
        np.add.at(out["dgate"], owner, t * n)
        np.add.at(mag["dgate"], owner, t_abs * np.abs(n))
    else:
        g = np.ones((1, 1))
    b, b_abs = t * g * w, t_abs * np.abs(g * w)
    if post_norm:
        out["dw_post"], mag["dw_post"] = np.sum(t * g * y * r, axis=0), np.sum(t_abs * np.abs(g * y * r), axis=0)
        out["dy"] = r * b - y * r**3 * np.mean(b * y, axis=1, keepdims=True)
        mag["dy"] = r * b_abs + np.abs(y) * r**3 * np.mean(b_abs * np.abs(y), axis=1, keepdims=True)
    else:
        out["dy"], mag["dy"] = b, b_abs
    return out, mag


def token_logps(logits, labels):
    """Log-probability of each label; 0 where the label is outside the vocabulary."""
    x = logits.astype(F).reshape(-1, logits.shape[-1])
    lab = labels.reshape(-1)
    out = np.zeros(lab.shape)
    for i, k in enumerate(lab):
        if 0 <= k < x.shape[1]:
            m = np.max(x[i])
            with np.errstate(invalid="ignore"):
                out[i] = x[i, k] - m - np.log(np.sum(np.exp(x[i] - m)))
    return out.reshape(labels.shape)


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def preference_loss(logits, labels, ref, beta, smoothing=0.0, grad_scale=1.0):
    """(loss, log_ratios [2P], logps [2P, S], dlogits [2P, S, V], coefficients [2P])."""
    n, S, V = logits.shape
    P = n // 2
    counted = (labels >= 0) & (labels < V)
    logps = token_logps(logits, labels)
    D = np.sum(np.where(counted, logps - (0.0 if ref is None else ref.astype(F)), 0.0), axis=1)
    z = beta * (D[:P] - D[P:])
    loss = np.mean((1 - smoothing) * softplus(-z) + smoothing * softplus(z))
    sig = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
    c = grad_scale * beta / P * (sig + smoothing - 1)
    c = np.concatenate([c, -c])
    d = np.zeros(logits.shape)
    for i in range(n):
        for t in range(S):
            if counted[i, t]:
                x = logits[i, t].astype(F)
                e = np.exp(x - np.max(x))
                d[i, t] = -c[i] * e / np.sum(e)
                d[i, t, labels[i, t]] += c[i]
    return loss, D, logps, d, c


def grad_norm(tensors):
    return float(np.sqrt(sum(float(np.sum(t.astype(F) ** 2)) for t in tensors)))


def clip_coefficient(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6))
