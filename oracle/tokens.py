"""Float64 oracle of the token-matrix operators: 8-bit quantization, the 8-bit
product, the root-mean-square norm and the distillation loss, each with its
gradient where it has one.  Written from the formulas; shares no code with
the CUDA path."""
from __future__ import annotations

import numpy as np


def quantize(x):
    """(q, scale) per row: scale = max|x| / 127, q = x / scale before rounding
    (the caller judges the rounding); a zero row has scale 0 and zeros."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.max(np.abs(x), axis=1, initial=0.0)
    scale = amax / 127.0
    q = np.divide(x, scale[:, None], out=np.zeros_like(x), where=scale[:, None] > 0)
    return q, scale


def int8_matmul(a, a_scale, b, b_scale):
    acc = np.asarray(a, dtype=np.int64) @ np.asarray(b, dtype=np.int64).T
    return acc.astype(np.float64) * np.asarray(a_scale, np.float64)[:, None] * \
        np.asarray(b_scale, np.float64)[None, :]


def rms_norm(h, w, eps):
    """(y, rstd) of the rows of h."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * np.asarray(w, np.float64), rstd


def rms_norm_grad(dy, h, w, rstd, dh=None):
    """(dx, dw)."""
    dy, h, w = (np.asarray(v, dtype=np.float64) for v in (dy, h, w))
    r = np.asarray(rstd, np.float64)[:, None]
    g = dy * w
    dx = r * (g - h * r * r * np.mean(g * h, axis=1, keepdims=True))
    if dh is not None:
        dx = dx + dh
    return dx, np.sum(dy * h * r, axis=0)


def teacher_probs(t, idx, vocab, tau):
    """Per row: (log p with -inf for what does not count, the valid mask)."""
    t = np.asarray(t, dtype=np.float64) / tau
    ok = (idx >= 0) & (idx < vocab) & (t != -np.inf)
    logp = np.full(t.shape, -np.inf)
    for r in range(t.shape[0]):
        v = t[r, ok[r]]
        if v.size:
            m = v.max()
            logp[r, ok[r]] = v - m - np.log(np.sum(np.exp(v - m)))
    return logp, ok


def distill_loss(s, t, idx, tau):
    """(loss, lse) per row."""
    s = np.asarray(s, dtype=np.float64) / tau
    logp, ok = teacher_probs(t, idx, s.shape[1], tau)
    loss, lse = np.zeros(s.shape[0]), np.zeros(s.shape[0])
    for r in range(s.shape[0]):
        if not ok[r].any():
            continue
        m = s[r].max()
        lse[r] = m + np.log(np.sum(np.exp(s[r] - m)))
        for k in np.nonzero(ok[r])[0]:
            p = np.exp(logp[r, k])
            if p > 0:
                loss[r] += p * (logp[r, k] - (s[r, idx[r, k]] - lse[r]))
    return loss * tau * tau, lse


def distill_grad(s, t, idx, lse, dloss, tau):
    """dS."""
    s = np.asarray(s, dtype=np.float64) / tau
    logp, ok = teacher_probs(t, idx, s.shape[1], tau)
    out = np.zeros(s.shape)
    for r in range(s.shape[0]):
        if not ok[r].any() or dloss[r] == 0:
            continue
        out[r] = np.exp(s[r] - float(lse[r]))
        for k in np.nonzero(ok[r])[0]:
            out[r, idx[r, k]] -= np.exp(logp[r, k])
        out[r] *= float(dloss[r]) * tau
    return out
