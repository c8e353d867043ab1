"""The operators of a replica in 64 bits: layer norm, linear layer and
distillation loss, forward and backward, each written from its definition.

Everything takes and returns float64 arrays; what the library rounds (its
inputs' type, the saved statistics) the caller rounds before the call.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erf, logsumexp


# ------------------------------------------------------------ layer norm

def norm_forward(x, gamma, beta, eps):
    """(y, mean, rstd)."""
    mean = x.mean(1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * gamma + beta, mean, rstd


def norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta)."""
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    n = x.shape[1]
    dx = rstd[:, None] * (g - g.sum(1, keepdims=True) / n - xh * (g * xh).sum(1, keepdims=True) / n)
    return dx, (dy * xh).sum(0), dy.sum(0)


# ------------------------------------------------------------ linear layer

def activation(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "gelu":
        return z * 0.5 * (1 + erf(z / np.sqrt(2)))
    if act == "gelu_tanh":
        return z * 0.5 * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + np.exp(-z))
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * (1 + erf(z / np.sqrt(2))) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if act == "gelu_tanh":
        c = np.sqrt(2 / np.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    return np.ones_like(z)


def linear_forward(x, w, bias, residual, act):
    """(y, z)."""
    z = x @ w.T + (0 if bias is None else bias)
    return activation(z, act) + (0 if residual is None else residual), z


def linear_backward(dy, z, x, w, act):
    """(dx, dw, dbias)."""
    dz = dy if act == "none" else dy * slope(z, act)
    return dz @ w, dz.T @ x, dz.sum(0)


# ------------------------------------------------------------ distillation

def _row(logits, teacher, index, T):
    """(kept, p, log p, log q at every entry of the vocabulary) of one row; a NaN logit of the teacher's is kept."""
    kept = (index >= 0) & (index < logits.size) & ~(teacher == -np.inf)
    t = teacher[kept]
    t = (t - t.max(initial=-np.inf)) / T
    logp = t - logsumexp(t) if t.size else t
    # relative to the largest logit: a common part of 1e38 would swallow the logarithm even in 64 bits
    shifted = (logits - logits.max()) / T
    return kept, np.exp(logp), logp, shifted - logsumexp(shifted)


def distill_forward(logits, teacher, index, T):
    """(loss, stats)."""
    loss, stats = np.zeros(len(logits)), np.zeros((len(logits), 2))
    for r, s in enumerate(logits):
        kept, p, logp, logq = _row(s, teacher[r], index[r], T)
        if kept.any():
            terms = [a * (b - c) if a else 0.0 for a, b, c in zip(p, logp, logq[index[r][kept]])]
            loss[r] = T * T * np.sum(terms)
            stats[r] = s.max(), np.log(np.sum(np.exp((s - s.max()) / T)))
    return loss, stats


def distill_backward(logits, teacher, index, dloss, T):
    """dlogits."""
    out = np.zeros_like(logits)
    for r, s in enumerate(logits):
        kept, p, _, logq = _row(s, teacher[r], index[r], T)
        if kept.any():
            out[r] = np.exp(logq)
            np.subtract.at(out[r], index[r][kept], p)
            out[r] *= dloss[r] * T
    return out
