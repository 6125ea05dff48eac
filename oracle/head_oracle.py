"""Reference (oracle) of the language-model head's row operators -- TEST INFRASTRUCTURE ONLY.

Plain numpy in fp64, one row at a time where that is clearer. Only the test suite uses this
module; no product path imports it. Logits come as fp64 arrays holding the exact values of
the bf16 or fp32 logits.

Conventions (include/prune24.h): a logit of -inf has probability 0 and gradient 0; a row of
nothing else has no distribution (log probabilities -inf, entropy 0, losses +inf where
anything is asked of it, gradients 0); tokens, labels and list entries outside 0..V-1 are
absent.
"""
from __future__ import annotations

import numpy as np


def _softmax_parts(z, tau):
    """m, ln s, x = (z - m) / tau of one row (m = -inf: ln s = -inf, x all -inf)."""
    m = z.max()
    if m == -np.inf:
        return m, -np.inf, np.full(z.shape, -np.inf)
    x = (z - m) / tau
    return m, np.log(np.exp(x).sum()), x


def order(z):
    """Columns of a row in falling order: NaN above +inf, -0 equal to +0, ties to the lower column."""
    rank = np.where(np.isnan(z), np.inf, np.where(z == np.inf, np.finfo(np.float64).max, z))
    return np.argsort(-rank, kind="stable")


def token_logprobs(Z, tokens=None, k=0, tau=1.0):
    T, V = Z.shape
    out = {"stats": np.zeros((T, 2)), "entropy": np.zeros(T), "top_logp": np.full((T, k), -np.inf),
           "top_idx": np.full((T, k), -1, dtype=np.int64)}
    if tokens is not None:
        out["logp"] = np.zeros(T)
    for t in range(T):
        z = Z[t]
        if np.isnan(z).any() or (z == np.inf).any():
            lp, h, st = np.full(V, np.nan), np.nan, (np.nan, np.nan)
        else:
            m, ls, x = _softmax_parts(z, tau)
            lp = x - ls if m > -np.inf else np.full(V, -np.inf)
            some = lp > -np.inf
            h, st = -(np.exp(lp[some]) * lp[some]).sum(), (m, ls)
        out["stats"][t], out["entropy"][t] = st, h
        if tokens is not None and 0 <= tokens[t] < V:
            out["logp"][t] = lp[tokens[t]]
        best = order(z)[:k]
        out["top_idx"][t, :len(best)] = best
        out["top_logp"][t, :len(best)] = lp[best]
    return out


def token_logprobs_bwd(Z, tokens, dlogp=None, dentropy=None, tau=1.0):
    T, V = Z.shape
    D = np.zeros((T, V))
    for t in range(T):
        m, ls, x = _softmax_parts(Z[t], tau)
        if m == -np.inf:
            continue
        lp = x - ls
        p = np.exp(lp)
        some = p > 0
        if dlogp is not None and 0 <= tokens[t] < V:
            D[t] -= dlogp[t] * p
            D[t, tokens[t]] += dlogp[t]
        if dentropy is not None:
            h = -(p[some] * lp[some]).sum()
            D[t, some] -= dentropy[t] * p[some] * (lp[some] + h)
    return D / tau


def teacher(idx, val, V, tau, tail):
    """Columns, probabilities and the remaining bucket's probability of one row's list."""
    on = (idx >= 0) & (idx < V)
    cols, v = idx[on], val[on].astype(np.float64)
    if tail:
        q = np.exp(v)
        return cols, q, max(0.0, 1.0 - q.sum())
    if len(v) == 0 or v.max() == -np.inf:
        return cols, np.zeros(len(v)), 0.0
    e = np.exp((v - v.max()) / tau)
    return cols, e / e.sum(), 0.0


def distill(Z, idx, val, labels=None, tau=1.0, tail=False, dkl=None, dce=None):
    """kl, ce, stats and (for weights dkl, dce) the gradient D."""
    T, V = Z.shape
    kl, ce, stats, D = np.zeros(T), np.zeros(T), np.zeros((T, 4)), np.zeros((T, V))
    for t in range(T):
        z = Z[t]
        m, ls, x = _softmax_parts(z, tau)
        none = m == -np.inf
        lp = np.full(V, -np.inf) if none else x - ls
        p = np.exp(lp)
        cols, q, q_rest = teacher(idx[t], val[t], V, tau, tail)
        off = np.ones(V, dtype=bool)
        off[cols] = False
        some = q > 0
        kl[t] = (q[some] * (np.log(q[some]) - lp[cols[some]])).sum()
        lr = 0.0
        if tail:
            rest = np.exp(x[off]).sum()
            lr = np.log(rest) if rest > 0 else -np.inf
            if rest == 0:
                q_rest = 0.0        # a bucket in which the student can have nothing is dropped
            if q_rest > 0:
                kl[t] += q_rest * (np.log(q_rest) - (lr - ls))
        l1 = 0.0
        has = labels is not None and 0 <= labels[t] < V
        if labels is not None:
            l1 = -np.inf if none else np.log(np.exp(z - m).sum())
        if has:
            ce[t] = np.inf if none else l1 - (z[labels[t]] - m)
        stats[t] = m, ls, lr, l1
        if none:
            continue
        if dkl is not None:
            total = q.sum() + q_rest
            g = total * p
            if q_rest > 0:
                g[off] = p[off] * (total - q_rest / np.exp(lr - ls))
            g[cols] -= q
            D[t] += dkl[t] / tau * g
        if dce is not None and has:
            D[t] += dce[t] * np.exp(z - m - l1)
            D[t, labels[t]] -= dce[t]
    return {"kl": kl, "ce": ce, "stats": stats, "dlogits": D}
