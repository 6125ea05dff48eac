"""Reference (oracle) of the operators around the sparse FFN (RMS norm, embedding, gradient norm) -- TEST
INFRASTRUCTURE ONLY.

Plain numpy in fp64 on arrays that hold the exact values of the bf16 or fp32 inputs. Only the test suite
uses this module; no product path imports it.

Conventions (include/prune24.h): the residual sum is rounded to the residual's type before the norm; a token
outside 0..V-1 is padding (a row of zeros, no gradient); a gradient norm that is not finite scales nothing.
"""
from __future__ import annotations

import numpy as np


def round_bf16(a):
    """The nearest bf16, ties to even, of fp64 values (one rounding)."""
    a = np.asarray(a, dtype=np.float64)
    out = a.copy()
    fin = np.isfinite(a) & (a != 0)
    e = np.maximum(np.frexp(a[fin])[1], -125)   # |a| in [2^(e-1), 2^e); below 2^-126 the step stays
    step = np.ldexp(1.0, e - 8)
    v = np.round(a[fin] / step) * step          # numpy rounds halves to even
    top = np.ldexp(255.0, 120)                  # the largest finite value
    out[fin] = np.where(np.abs(v) > top, np.copysign(np.inf, v), v)
    return out


def round_f32(a):
    with np.errstate(over="ignore"):
        return np.asarray(a, dtype=np.float64).astype(np.float32).astype(np.float64)


def e4m3_value(code):
    """The value of a code: sign, 4 exponent bits (bias 7), 3 fraction bits; no infinities, 0x7f is NaN."""
    s, e, f = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and f == 7:
        return np.nan
    v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
    return -v if s else v


_CODES = np.array([e4m3_value(c) for c in range(127)])  # rising, 0 to 448


def round_e4m3(v):
    """The nearest value that a code has, ties to the even code, magnitudes above 448 to 448."""
    v = np.asarray(v, dtype=np.float64)
    m = np.minimum(np.abs(v), 448.0)
    hi = np.clip(np.searchsorted(_CODES, m), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - _CODES[lo], _CODES[hi] - m
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(v), np.nan, np.copysign(_CODES[pick], v))


def rmsnorm(x, w=None, r=None, eps=1e-6, rounded=None):
    """h, rstd, y (unrounded); rounded: the rounding of the residual's type."""
    h = x if r is None else rounded(x + r)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        rstd = 1 / np.sqrt((h * h).mean(1) + eps)
        y = h * rstd[:, None] * (1.0 if w is None else w)
    return h, rstd, y


def scales(y, group):
    """Per row and group of columns: the largest magnitude / 448; 1 for a group of zeros."""
    d = y.shape[1]
    group = group or d
    out = np.stack([np.abs(y[:, c:c + group]).max(1) for c in range(0, d, group)], 1) / 448
    return np.where(out == 0, 1.0, np.maximum(out, 2.0 ** -118))


def spread(s, d, group):
    return np.repeat(s, group or d, axis=1)[:, :d]


def rmsnorm_bwd(dy, h, w, eps=1e-6, dres=None):
    """dx and dweight, the gradients of sum(y dy) + sum(h dres)."""
    rstd = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    xh = h * rstd
    g = dy * (1.0 if w is None else w)
    dx = rstd * (g - xh * (g * xh).mean(1, keepdims=True))
    return dx + (0 if dres is None else dres), (dy * xh).sum(0)


def embed(tokens, W, scale=1.0):
    out = np.zeros((len(tokens), W.shape[1]))
    for t, v in enumerate(tokens):
        if 0 <= v < W.shape[0]:
            out[t] = scale * W[v]
    return out


def embed_bwd(dY, tokens, V, scale=1.0, dW=None):
    out = np.zeros((V, dY.shape[1])) if dW is None else dW.copy()
    for t, v in enumerate(tokens):
        if 0 <= v < V:
            out[v] += scale * dY[t]
    return out


def grad_norm(grads):
    return np.sqrt(sum(float(np.square(g, dtype=np.float64).sum()) for g in grads))


def clip(grads, max_norm):
    n = grad_norm(grads)
    f = max_norm / n if np.isfinite(n) and n > max_norm else 1.0
    return n, [g * f for g in grads]
