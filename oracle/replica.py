"""The operators of a replica in 64 bits: layer norm, linear layer,
distillation loss, dropout, RMS norm and the log probabilities of tokens,
forward and backward, each written from its definition.

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


# ------------------------------------------------------------ dropout

def philox(key, counter, stream):
    """The four 32-bit words of Philox4x32-10 (Salmon et al., 2011), in Python integers."""
    low = (1 << 32) - 1
    k = [key & low, key >> 32 & low]
    c = [counter & low, counter >> 32 & low, stream & low, stream >> 32 & low]
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [q >> 32 ^ c[1] ^ k[0], q & low, p >> 32 ^ c[3] ^ k[1], p & low]
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    return c


def dropout_mask(rows, cols, p, seed, offset, first_row):
    """(kept, scale)."""
    drop, per = int(p * 65536 + 0.5), -(-cols // 8)
    kept = np.zeros((rows, per * 8), bool)
    for r in range(rows):
        for n in range(per):
            words = philox(seed, (first_row + r) * per + n, offset)
            for e in range(8):
                kept[r, 8 * n + e] = (words[e // 2] >> 16 * (e % 2) & 0xFFFF) >= drop
    return kept[:, :cols], 65536 / (65536 - drop) if drop < 65536 else 0.0


def dropout(x, residual, p, seed, offset=0, first_row=0):
    kept, scale = dropout_mask(*x.shape, p, seed, offset, first_row)
    return np.where(kept, x * scale, 0.0) + residual


# ------------------------------------------------------------ RMS norm

def rms_forward(s, gamma, eps):
    """(y, rstd) of the sum s."""
    rstd = 1 / np.sqrt((s ** 2).mean(1) + eps)
    return s * rstd[:, None] * gamma, rstd


def rms_backward(dy, dsum, s, gamma, rstd):
    """(dx, dgamma)."""
    xh, g = s * rstd[:, None], dy * gamma
    dx = dsum + rstd[:, None] * (g - xh * (g * xh).sum(1, keepdims=True) / s.shape[1])
    return dx, (dy * xh).sum(0)


def group_scales(y, quant, group):
    """[rows, groups]: the largest |y| of each group of columns over the largest code."""
    group = group or y.shape[1]
    most = np.stack([np.abs(y[:, at:at + group]).max(1) for at in range(0, y.shape[1], group)], 1)
    return np.maximum(most / {"int8": 127.0, "e4m3": 448.0}[quant], 2.0 ** -126)


# ------------------------------------------------------------ log probabilities of tokens

def _logq(s, T):
    """log softmax(s / T) of one row, or None where all of it is -inf."""
    if s.size == 0 or (s == -np.inf).all():
        return None
    x = (s - s.max()) / T
    return x - logsumexp(x)


def logprob_forward(logits, token, k, T):
    """(logprob, entropy, stats, top, index); a token of None: none are given."""
    n, vocab = logits.shape
    logprob, entropy, stats = np.zeros(n), np.zeros(n), np.zeros((n, 2))
    top, index = np.full((n, k), -np.inf), np.full((n, k), -1)
    for r, s in enumerate(logits):
        if token is not None and not 0 <= token[r] < vocab:
            continue
        logq = _logq(s, T)
        if logq is None:
            stats[r], logprob[r] = (-np.inf, 0), -np.inf
            logq = np.full(vocab, -np.inf)
        else:
            q = np.exp(logq)
            entropy[r] = -np.sum(np.where(q > 0, q * np.where(q > 0, logq, 0), 0.0 if not np.isnan(q).any() else np.nan))
            logprob[r] = logq[token[r]] if token is not None else 0
            with np.errstate(invalid="ignore"):
                stats[r] = s.max(), np.log(np.sum(np.exp((s - s.max()) / T)))
        if k == 0:
            continue
        nan = np.isnan(s)
        order = np.lexsort((np.arange(vocab), np.where(nan, 0, -s), ~nan))[:k]  # NaN first, the largest, the lowest index
        top[r, :len(order)], index[r, :len(order)] = logq[order], order
    return logprob, entropy, stats, top, index


def logprob_backward(logits, token, dlogprob, dentropy, T):
    """dlogits."""
    out = np.zeros_like(logits)
    for r, s in enumerate(logits):
        logq = _logq(s, T)
        if logq is None or (token is not None and not 0 <= token[r] < s.size):
            continue
        q, known = np.exp(logq), np.where(np.exp(logq) > 0, logq, 0)
        out[r] = -dlogprob[r] * q - dentropy[r] * q * (known - np.sum(q * known))
        if token is not None:
            out[r, token[r]] += dlogprob[r]
        out[r] /= T
    return out
