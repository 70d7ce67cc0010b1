"""fp64 oracle of the residual RMS norm, the scored router, and FP8 with one scale per block of 128.

Written from the operators' definitions; imports nothing from the package."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from .mx import POS_VALUES

FP8_MAX = 448.0
TINY = 2.0 ** -100


# ------------------------------------------------------------------ norm
def add_rmsnorm(h, w, eps):
    """(y, rstd) of rows h (the rounded sum x + residual)."""
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def add_rmsnorm_backward(dy, dh, h, w, rstd):
    """(dx, dw); dh may be None."""
    xh = h * rstd[:, None]
    q = dy * w
    dx = rstd[:, None] * (q - xh * np.mean(q * xh, axis=1, keepdims=True))
    return (dx if dh is None else dh + dx), np.sum(dy * xh, axis=0)


# ------------------------------------------------------------------ scored routing
@dataclass(frozen=True)
class Rule:
    score: str = "softmax"
    groups: int = 1
    top_groups: int = 1
    group_top: int = 1
    renormalise: bool = True
    scale: float = 1.0


def scores(l, rule):
    if rule.score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    m = np.max(l, axis=1, keepdims=True)
    p = np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isneginf(m), 0.0, m)))
    tot = p.sum(axis=1, keepdims=True)
    return np.divide(p, tot, out=np.zeros_like(p), where=tot > 0)


def _best(v, n):
    """The n largest of v, ties to the lower index."""
    return np.lexsort((np.arange(v.size), -v))[:n]


def choose(l, rule, k, balance=None):
    """Expert ids [T, k] ascending, one token at a time."""
    s = scores(l, rule)
    c = s if balance is None else s + balance
    T, E = l.shape
    per = E // rule.groups
    out = np.empty((T, k), dtype=np.int64)
    for t in range(T):
        group = np.array([np.sort(c[t, g * per:(g + 1) * per])[::-1][:rule.group_top].sum() for g in range(rule.groups)])
        kept = _best(group, rule.top_groups)
        ids = np.concatenate([np.arange(g * per, (g + 1) * per) for g in np.sort(kept)])
        order = l[t] if balance is None else c[t]
        out[t] = np.sort(ids[_best(order[ids], k)])
    return out


def margins(l, rule, k, balance=None):
    """How far each token's choice is from a tie (in units of c, and of l where that decides)."""
    s = scores(l, rule)
    c = s if balance is None else s + balance
    T, E = l.shape
    per = E // rule.groups
    out = np.full(T, np.inf)
    for t in range(T):
        group = np.sort([np.sort(c[t, g * per:(g + 1) * per])[::-1][:rule.group_top].sum() for g in range(rule.groups)])[::-1]
        if rule.top_groups < rule.groups:
            out[t] = group[rule.top_groups - 1] - group[rule.top_groups]
        kept = _best(np.array([np.sort(c[t, g * per:(g + 1) * per])[::-1][:rule.group_top].sum() for g in range(rule.groups)]),
                     rule.top_groups)
        ids = np.concatenate([np.arange(g * per, (g + 1) * per) for g in kept])
        v = np.sort((l[t] if balance is None else c[t])[ids])[::-1]
        if k < v.size:
            out[t] = min(out[t], v[k - 1] - v[k])
    return out


def gates(l, idx, rule):
    s = np.take_along_axis(scores(l, rule), idx, axis=1)
    if rule.renormalise:
        tot = s.sum(axis=1, keepdims=True)
        s = np.divide(s, tot, out=np.zeros_like(s), where=tot > 0)
    return rule.scale * s


def gates_backward(dg, l, idx, rule):
    """dl [T, E] of the gates."""
    s = scores(l, rule)
    ds = np.zeros_like(s)
    dg = rule.scale * dg
    if rule.renormalise:
        sk = np.take_along_axis(s, idx, axis=1)
        tot = sk.sum(axis=1, keepdims=True)
        inner = np.divide((dg * sk).sum(axis=1, keepdims=True), tot, out=np.zeros_like(tot), where=tot > 0)
        dg = np.divide(dg - inner, tot, out=np.zeros_like(dg), where=tot > 0)
    for t in range(l.shape[0]):
        for j in range(idx.shape[1]):
            ds[t, idx[t, j]] += dg[t, j]
    if rule.score == "sigmoid":
        with np.errstate(over="ignore"):
            return ds * s / (1.0 + np.exp(l))
    if rule.renormalise:   # sum_e ds s = 0: the gates do not see what is outside S
        return s * ds
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))


# ------------------------------------------------------------------ FP8
def e4m3(v):
    """Nearest E4M3 value, ties to the even code, saturating (a search among the format's values)."""
    a = np.minimum(np.abs(np.asarray(v, dtype=np.float64)), FP8_MAX)
    hi = np.searchsorted(POS_VALUES, a, side="left")
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - POS_VALUES[lo], POS_VALUES[hi] - a
    pick = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(POS_VALUES[pick], v)


def quantise_rows(x):
    """(values of the codes [M, K], scales [M, K / 128])."""
    M, K = x.shape
    b = x.reshape(M, K // 128, 128)
    s = np.maximum(np.abs(b).max(axis=2), TINY) / FP8_MAX
    return e4m3(b / s[:, :, None]).reshape(M, K), s


def quantise_blocks(w):
    """(values of the codes [N, K], scales [ceil(N / 128), K / 128])."""
    N, K = w.shape
    s = np.empty((-(-N // 128), K // 128))
    q = np.empty_like(w)
    for r in range(s.shape[0]):
        for c in range(s.shape[1]):
            b = w[128 * r:128 * r + 128, 128 * c:128 * c + 128]
            s[r, c] = max(np.abs(b).max(), TINY) / FP8_MAX
            q[128 * r:128 * r + 128, 128 * c:128 * c + 128] = e4m3(b / s[r, c])
    return q, s


def spread_rows(q, s):
    return q * np.repeat(s, 128, axis=1)


def spread_blocks(q, s):
    return q * np.repeat(np.repeat(s, 128, axis=0)[:q.shape[0]], 128, axis=1)


def expert_ffn(x, wg, wu, wd):
    """Y of one expert's rows (all operands spread to values): (y, a, u), H quantised per 1 x 128."""
    a, u = x @ wg.T, x @ wu.T
    with np.errstate(over="ignore"):
        h = a / (1.0 + np.exp(-a)) * u
    return spread_rows(*quantise_rows(h)) @ wd.T, a, u
