"""Float64 definitions of the operators of a training step around the adapter
linears (numpy): embedding lookup and gradient, token log probabilities, the
preference and policy losses with their derivatives, the gradient of the
logits, AdamW and its 8-bit states. Every input converts to float64 exactly;
nothing is blocked, fused or rounded."""
from __future__ import annotations

import numpy as np

E4M3_MAX, E4M3_MIN, STATE_BLOCK = 448.0, 2.0 ** -9, 256


def _f64(a):
    return np.asarray(a, np.float64)


def embed(ids, table, scale):
    ids, table = np.asarray(ids), _f64(table)
    out = np.zeros((len(ids), table.shape[1]))
    ok = (ids >= 0) & (ids < len(table))
    out[ok] = scale * table[ids[ok]]
    return out


def embed_grad(ids, dy, rows, scale, old=None):
    ids, dy = np.asarray(ids), _f64(dy)
    out = np.zeros((rows, dy.shape[1])) if old is None else _f64(old).copy()
    for t, v in enumerate(ids):
        if 0 <= v < rows:
            out[v] += scale * dy[t]
    return out


def masked(targets, vocab):
    targets = np.asarray(targets)
    return (targets < 0) | (targets >= vocab)


def token_logp(logits, targets):
    x, y = _f64(logits), np.asarray(targets)
    off = masked(y, x.shape[1])
    out = np.zeros(len(x))
    for t in np.flatnonzero(~off):
        with np.errstate(all="ignore"):
            m = x[t].max()
            out[t] = (x[t, y[t]] - m) - np.log(np.exp(x[t] - m).sum())
    return out


def softmax(logits):
    x = _f64(logits)
    with np.errstate(all="ignore"):
        e = np.exp(x - x.max(1, keepdims=True)) if x.shape[1] else x
        return e / e.sum(1, keepdims=True)


def logit_grad(logits, targets, coef):
    x, y = _f64(logits), np.asarray(targets)
    out = -softmax(x)
    off = masked(y, x.shape[1])
    live = np.flatnonzero(~off)
    out[live, y[live]] += 1.0
    out *= _f64(coef)[:, None]
    out[off] = 0.0
    return out


def _log_sigmoid(z):
    return -np.logaddexp(0.0, -z)


def pref_loss(logp, offsets, ref, beta, eps):
    """(loss, seq_logp, d loss / d logp)"""
    logp, ref = _f64(logp), _f64(ref)
    T, n = len(logp), len(ref)
    o = np.clip(np.asarray(offsets, np.int64), 0, T)
    seq = np.array([logp[o[s]:o[s + 1]].sum() for s in range(n)])
    coef = np.zeros(T)
    loss = 0.0
    for p in range(n // 2):
        c, r = 2 * p, 2 * p + 1
        z = beta * ((seq[c] - ref[c]) - (seq[r] - ref[r]))
        loss += -(1 - eps) * _log_sigmoid(z) - eps * _log_sigmoid(-z)
        d = beta * (-(1 - eps) * np.exp(_log_sigmoid(-z)) + eps * np.exp(_log_sigmoid(z))) / (n // 2)
        coef[o[c]:o[c + 1]] = d
        coef[o[r]:o[r + 1]] = -d
    return loss / (n // 2), seq, coef


def policy_loss(logp, targets, vocab, old, adv, weights, low, high, ref=None, kl=0.0):
    """(loss, d loss / d logp)"""
    live = np.flatnonzero(~masked(targets, vocab))
    loss, coef = 0.0, np.zeros(len(_f64(logp)))
    for t in live:
        lp, a, w = float(logp[t]), float(adv[t]), float(weights[t])
        r = np.exp(lp - float(old[t]))
        held = min(max(r, 1 - low), 1 + high)
        term, d = (-r * a, -r * a) if r * a <= held * a else (-held * a, 0.0)
        if kl != 0.0:
            k = float(ref[t]) - lp
            term += kl * (np.exp(k) - k - 1)
            d += kl * (1 - np.exp(k))
        loss += w * term
        coef[t] = w * d
    return loss, coef


def adamw(p, g, m, v, t, lr, beta1, beta2, eps, decay):
    """(p, m, v) after the t-th step"""
    p, g, m, v = _f64(p), _f64(g), _f64(m), _f64(v)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = p - lr * decay * p - lr * (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p, m, v


def e4m3_step(x):
    """Spacing of the e4m3 values at |x|: 3 fraction bits, exponents from -6."""
    _, ex = np.frexp(np.abs(_f64(x)))
    return np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)


def quantise(x, positive):
    """(codes' values, scales) of blocks of 256 elements"""
    b = _f64(x).reshape(-1, STATE_BLOCK)
    amax = np.abs(b).max(1)
    scale = np.where(amax >= 1e-30, amax / E4M3_MAX, 0.0)
    q = b / np.where(scale > 0, scale, 1.0)[:, None] * (scale > 0)[:, None]
    code = np.round(q / e4m3_step(q)) * e4m3_step(q)
    if positive:
        code = np.where((q > 0) & (code == 0), E4M3_MIN, code)
    return code.reshape(-1), scale
