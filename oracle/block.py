"""fp64 oracle of the block norms, the 8-bit activation checkpoints and the draft verification.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The definitions as include/rlk.h states them.  Gradients are the formulas' own;
``tests/test_block_oracle.py`` checks them against central differences.
"""
from __future__ import annotations

import math

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


# ---------------------------------------------------------------- 8-bit checkpoints
E4M3 = np.array([(-1.0 if b & 0x80 else 1.0) * (((b & 7) + 8) * 2.0 ** ((b >> 3 & 15) - 10) if b >> 3 & 15
                                              else (b & 7) * 2.0 ** -9) for b in range(256)])


def quantize(x, fmt):
    """(codes uint8 [T, H], scales uint8 [T, H / 32]) of bf16 values given in fp64."""
    x = _f64(x)
    T, H = x.shape
    codes, scales = np.zeros((T, H), np.uint8), np.zeros((T, H // 32), np.uint8)
    finite = np.sort(E4M3[:0x7F])  # 0 .. 448
    for t in range(T):
        for k in range(H // 32):
            v = x[t, 32 * k:32 * k + 32]
            if not np.all(np.isfinite(v)):
                scales[t, k] = 255
                continue
            big = np.abs(v).max()
            e = max(math.frexp(big)[1] - 1, -127) if big > 0 else -127
            if fmt == "int8":
                b = e + 127
                q = np.clip(np.rint(v * 2.0 ** (133 - b)), -127, 127)  # rint: ties to even
                codes[t, 32 * k:32 * k + 32] = q.astype(np.int64) & 0xFF
            else:
                b = max(e + 119 + (1 if big > 1.75 * 2.0 ** e and e < 127 else 0), 0)
                u = np.minimum(np.abs(v) * 2.0 ** (127 - b), 448.0)
                lo = np.clip(np.searchsorted(finite, u, side="right") - 1, 0, 0x7E)
                hi = np.minimum(lo + 1, 0x7E)
                dl, dh = u - finite[lo], finite[hi] - u
                up = (dh < dl) | ((dh == dl) & (hi % 2 == 0) & (hi != lo))
                c = np.where(up, hi, lo)
                codes[t, 32 * k:32 * k + 32] = c | np.where(np.signbit(v), 0x80, 0)
            scales[t, k] = b
    return codes, scales


def dequantize(codes, scales, fmt):
    """The values, fp64."""
    s = np.repeat(scales.astype(np.float64), 32, axis=1)
    v = codes.view(np.int8) * 2.0 ** (s - 133) if fmt == "int8" else E4M3[codes] * 2.0 ** (s - 127)
    return np.where(s == 255, np.nan, v)


# ---------------------------------------------------------------- block norms
def _rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)


def gate_value(gate, kind):
    """(gate(g), gate'(g))"""
    if gate is None:
        return 1.0, 0.0
    gate = _f64(gate)
    if kind == "identity":
        return gate, np.ones_like(gate)
    e = np.exp(-np.abs(gate))
    return np.where(gate < 0, e, 1.0) / (1 + e), e / (1 + e) ** 2


def block_stream(block, residual, gamma_post=None, gate=None, kind="sigmoid", rs=1.0, bs=1.0, eps=1e-6):
    """(x' before its rounding, the branch's part of it)"""
    b, r = _f64(block), _f64(residual)
    n = b if gamma_post is None else b * _rms(b, eps) * _f64(gamma_post)
    t = bs * n * gate_value(gate, kind)[0]
    return rs * r + t, t


def _norm_backward(up, x, eps):
    rstd = _rms(x, eps)
    return rstd * (up - x * rstd ** 2 * (up * x).mean(axis=1, keepdims=True))


def block_backward(grad_out, x, gamma_pre, block=None, gamma_post=None, gate=None, kind="sigmoid", rs=1.0,
                   bs=1.0, eps=1e-6, grad_res=None):
    """dict of the gradients, and the intermediate values that the tolerances go by."""
    dy, x, gp, b, gq = _f64(grad_out), _f64(x), _f64(gamma_pre), _f64(block), _f64(gamma_post)
    dx = _norm_backward(dy * gp, x, eps)
    if grad_res is not None:
        dx = dx + _f64(grad_res)
    d = bs * dx
    g, slope = gate_value(gate, kind)
    out = dict(dx=dx, d=d, grad_residual=rs * dx, grad_gamma_pre=(dy * x * _rms(x, eps)).sum(0),
               grad_gate=None, grad_gamma_post=None)
    w = d * g
    if gate is not None:
        n = b if gq is None else b * _rms(b, eps) * gq
        out.update(n=n, slope=slope, gate=g, grad_gate=d * n * slope)
    if gq is None:
        out["grad_block"] = w
    else:
        out["grad_gamma_post"] = (w * b * _rms(b, eps)).sum(0)
        out["grad_block"] = _norm_backward(w * gq, b, eps)
    out["w"] = w
    return out


# ---------------------------------------------------------------- drafted tokens
def draft_verify(target, tokens, uniforms, noise, offsets, draft=None, draft_lse=None, active=None):
    """(accepted, tokens, logprob, margin): margin [S] is how far, relatively, a sequence's closest
    decision was from going the other way."""
    target, noise = _f64(target), _f64(noise)
    S, D = len(offsets) - 1, len(tokens)
    accepted = np.zeros(S, np.int64)
    out, logprob = np.full(D + S, -1, np.int64), np.zeros(D + S)
    margin = np.full(S, np.inf)
    for s in range(S):
        b, e = int(offsets[s]), int(offsets[s + 1])
        if active is not None and not active[s]:
            continue
        for i in range(e - b + 1):
            row = target[b + s + i]
            top = row.max()
            lse = top + math.log(np.exp(row - top).sum())
            p = np.exp(row - lse)
            at = b + s + i
            if i < e - b:
                x = int(tokens[b + i])
                if draft is None:
                    q = np.zeros_like(p)
                    q[x] = 1.0
                else:
                    q = np.exp(_f64(draft[b + i]) - (0.0 if draft_lse is None else float(draft_lse[b + i])))
                u = float(uniforms[b + i])
                if u * q[x] > 0 and p[x] > 0:
                    margin[s] = min(margin[s], abs(u * q[x] / p[x] - 1))
                if u * q[x] < p[x]:
                    out[at], logprob[at] = x, row[x] - lse
                    accepted[s] += 1
                    continue
                number = ~np.isnan(q)  # a token whose q is none is never drawn
                w = np.where(number, np.maximum(p - np.where(number, q, 0.0), 0.0), 0.0)
                if not (w > 0).any():
                    w = np.where(number, p, 0.0)
                if not (w > 0).any():
                    logprob[at] = np.nan
                    break
            else:
                w = p
            race = w / noise[s]
            v = int(np.argmax(race))  # the lowest of equals
            two = np.sort(race)[-2:] if race.size > 1 else np.array([0.0, race[0]])
            # w's own error, relative to p, weighs more where little of p is left
            margin[s] = min(margin[s], (1 - two[0] / two[1]) * w[v] / p[v])
            out[at], logprob[at] = v, row[v] - lse
            break
    return accepted, out, logprob, margin
