"""The router's choice by its scores, in 80-bit numbers and without rounding them to any grid: what the library's choice
is compared with where scores are small or close (numpy, no library code)."""

from __future__ import annotations

import numpy as np

import router_ref as R

FLOAT_MAX = float(np.finfo(np.float32).max)
LEAST = {True: -104.0, False: -690.0}  # the least exponent of a score, sigmoid and softmax


def scores(x, ok, sigmoid):
    """Scores of one token's logits in 80 bits, 0 where not eligible."""
    y = np.where(ok, np.minimum(np.where(ok, x, 0), np.finfo(np.float32).max), 0).astype(np.longdouble)
    if sigmoid:
        s = 1 / (1 + np.exp(-np.clip(y, LEAST[True], -LEAST[True])))
    else:
        e = np.where(ok, np.exp(np.maximum(y - np.max(y[ok], initial=-np.inf), LEAST[False])), 0)
        s = e / max(e.sum(), np.longdouble(1))
    return np.where(ok, s, np.longdouble(0))


def cut(v):
    """42 significant bits of a value, the rest cut off."""
    v = np.asarray(v, np.longdouble)
    m, e = np.frexp(np.where(np.isfinite(v), v, 0))
    return np.where(np.isfinite(v), np.ldexp(np.trunc(np.ldexp(m, 42)), e - 42), v)


def _ranked(values, count, gaps):
    """Indices of the `count` largest values above -inf, descending, ties to the lower index.  Notes the least relative
    difference between unequal values that stand next to each other in that order."""
    order = sorted(range(len(values)), key=lambda i: (-values[i], i))
    order = [i for i in order if values[i] > -np.inf]
    for a, b in zip(order[:count], order[1:]):
        if values[a] != values[b]:
            gaps.append(float((values[a] - values[b]) / max(abs(values[a]), abs(values[b]))))
    return order[:count]


def choose(x, k, sigmoid, bias=None, groups=1, keep=1, group_top=1, mask=None):
    """-> (idx int32 [bs, k], for each row the least relative difference that a comparison rested on)."""
    bs, e = x.shape
    size = e // groups
    idx = np.full((bs, k), -1, np.int32)
    least = np.ones(bs)
    ok_all = R.eligible(x, mask)
    for t in range(bs):
        ok = ok_all[t]
        gaps = [1.0]
        if not ok.any():
            continue
        b = np.zeros(e, np.longdouble) if bias is None else np.asarray(bias, np.longdouble)
        off = ~(b > -np.inf)
        with np.errstate(invalid="ignore"):
            u = cut(np.clip(scores(x[t], ok, sigmoid) + np.where(off, 0, b), -R.CLIP, R.CLIP))
        u = np.where(ok & ~off, u, -np.inf)
        v = u if bias is not None else np.where(ok, np.clip(np.where(ok, x[t], 0), -FLOAT_MAX, FLOAT_MAX), -np.inf)
        if groups > 1:
            best = []
            for g in range(groups):
                part = np.sort((v if group_top == 1 else u)[g * size:(g + 1) * size])[::-1][:group_top]
                part = part[part > -np.inf]
                best.append(cut(part.sum()) if len(part) else -np.inf)
            kept = _ranked(best, keep, gaps)
            v = np.where(np.isin(np.arange(e) // size, kept), v, -np.inf)
        at = _ranked(v, k, gaps)
        idx[t, :len(at)] = at
        least[t] = min(gaps)
    return idx, least
