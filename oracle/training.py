"""fp64 oracle of the training-step operators around the selected-token logprob.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The definitions, written with explicit loops over sequences and pairs: the
clipped policy loss with a KL term, the preference loss on paired log ratios,
the global gradient norm with clipping, and the backward of the RMSNorm.
Gradients are the formulas' own; ``tests/test_training_oracle.py`` checks them
against central differences of the losses.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def policy_loss(logprob, old, advantages, ref=None, active=None, offsets=None, per_seq=False,
                clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl="k3", kl_coef=0.0,
                reduction="token_mean", scale=1.0):
    """(loss, stats [4], grad [T], weights [T]) of the clipped policy loss."""
    lp, old, ref, adv = _f64(logprob), _f64(old), _f64(ref), _f64(advantages)
    T = lp.shape[0]
    offsets = [0, T] if offsets is None else [int(o) for o in offsets]
    S = len(offsets) - 1
    on = np.ones(T, bool) if active is None else np.asarray(active) != 0
    on = on.copy()
    on[:offsets[0]] = False
    on[offsets[-1]:] = False
    w = np.zeros(T)
    A = np.zeros(T)
    n_all = max(1, int(on.sum()))
    for s in range(S):
        b, e = offsets[s], offsets[s + 1]
        n = max(1, int(on[b:e].sum()))
        w[b:e] = {"sum": 1.0, "token_mean": 1.0 / n_all, "seq_mean": 1.0 / (S * n)}[reduction]
        A[b:e] = adv[s] if per_seq else adv[b:e]
    grad = np.zeros(T)
    stats = np.zeros(4)
    for t in np.nonzero(on)[0]:
        d = lp[t] - old[t]
        r = math.exp(d)
        clipped = min(max(r, 1.0 - clip_low), 1.0 + clip_high)
        s, slope, shut = r * A[t], r * A[t], False
        if clipped * A[t] < s:
            s, slope, shut = clipped * A[t], 0.0, True
        if dual_clip > 0 and A[t] < 0 and dual_clip * A[t] > s:
            s, slope, shut = dual_clip * A[t], 0.0, True
        k = dk = 0.0
        if ref is not None:
            u = lp[t] - ref[t]
            k, dk = {"k1": (u, 1.0), "k2": (u * u / 2, u),
                     "k3": (math.expm1(-u) + u, -math.expm1(-u))}[kl]
        grad[t] = scale * w[t] * (-slope + kl_coef * dk)
        stats += w[t] * np.array([-s, k, float(shut), -d])
    return scale * (stats[0] + kl_coef * stats[1]), stats, grad, np.where(on, w, 0.0)


def preference_loss(logprob, offsets, ref=None, active=None, beta=0.1, kind="sigmoid",
                    label_smoothing=0.0, margin=0.0, length_normalize=False, layout="adjacent",
                    scale=1.0):
    """(loss, pair_loss [P], rewards [2P], grad [T], z [P]) of the preference loss."""
    lp, ref = _f64(logprob), _f64(ref)
    T = lp.shape[0]
    offsets = [int(o) for o in offsets]
    S = len(offsets) - 1
    P = S // 2
    on = np.ones(T, bool) if active is None else np.asarray(active) != 0
    m, n = np.zeros(S), np.ones(S)
    for s in range(S):
        at = [t for t in range(offsets[s], offsets[s + 1]) if on[t]]
        m[s] = math.fsum(lp[t] - (0.0 if ref is None else ref[t]) for t in at)
        if length_normalize:
            n[s] = max(1, len(at))
            m[s] /= n[s]
    pair_loss, zs, grad = np.zeros(P), np.zeros(P), np.zeros(T)

    def log_sig(v):
        return -(math.log1p(math.exp(-abs(v))) + max(-v, 0.0))

    for i in range(P):
        c, r = (2 * i, 2 * i + 1) if layout == "adjacent" else (i, P + i)
        h = m[c] - m[r]
        z = beta * h - margin
        zs[i] = z
        if kind == "sigmoid":
            pair_loss[i] = -(1 - label_smoothing) * log_sig(z) - label_smoothing * log_sig(-z)
            dh = beta * (label_smoothing * math.exp(log_sig(z))
                         - (1 - label_smoothing) * math.exp(log_sig(-z)))
        elif kind == "hinge":
            pair_loss[i] = max(0.0, 1.0 - z)
            dh = -beta if z < 1.0 else 0.0
        else:
            pair_loss[i] = (h - 0.5 / beta) ** 2
            dh = 2 * (h - 0.5 / beta)
        for s, sign in ((c, 1.0), (r, -1.0)):
            b, e = offsets[s], offsets[s + 1]
            grad[b:e] = np.where(on[b:e], sign * scale / P * dh / n[s], 0.0)
    loss = scale * pair_loss.mean() if P else 0.0
    return loss, pair_loss, beta * m, grad, zs


def clip_scale(grads: Sequence[np.ndarray], max_norm: float) -> Tuple[float, float]:
    """(norm, scale) of the global gradient norm's clipping."""
    norm = math.sqrt(math.fsum(float(np.sum(_f64(g) ** 2)) for g in grads))
    if math.isfinite(norm) and norm > max_norm:
        return norm, max_norm / norm
    return norm, 1.0


def rmsnorm_backward(grad_out, x, gamma, eps: float, grad_residual: Optional[np.ndarray] = None):
    """(grad_x [T, H], grad_gamma [H]) of y = x / sqrt(mean(x^2) + eps) * gamma."""
    dy, x, gamma = _f64(grad_out), _f64(x), _f64(gamma)
    H = x.shape[1]
    rstd = 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)
    up = dy * gamma
    c = rstd ** 2 / H * (up * x).sum(axis=1, keepdims=True)
    grad_x = rstd * (up - x * c)
    if grad_residual is not None:
        grad_x = grad_x + _f64(grad_residual)
    return grad_x, (dy * x * rstd).sum(axis=0)
