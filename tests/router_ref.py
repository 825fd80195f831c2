"""Plain 64-bit definitions of the router, its gradient, the combine's
gradient and the scaled expert product (numpy, no library code), and the
inputs their tests share."""

from __future__ import annotations

import numpy as np

GRID, CLIP = 2.0 ** 30, 1024.0
U = 2.0 ** -24  # half a step of binary32, relative


def eligible(x, mask=None):
    ok = np.nan_to_num(x, nan=-np.inf, posinf=np.inf, neginf=-np.inf) > -np.inf
    return ok if mask is None else ok & (np.asarray(mask) != 0)[:, None]


def scores(x, ok, sigmoid):
    """Scores of one token's logits (1-D, 64 bits); 0 where not eligible."""
    s = np.zeros(len(x))
    if not ok.any():
        return s
    y = np.minimum(x[ok], np.finfo(np.float32).max)
    with np.errstate(over="ignore", under="ignore"):
        if sigmoid:
            e = np.exp(-np.abs(y))
            s[ok] = np.where(y > 0, 1, e) / (1 + e)
        else:
            e = np.exp(y - y.max())
            s[ok] = e / e.sum()
    return s


def shares(y, sigmoid):
    """s / sum(s) of chosen logits (all finite), where the scores may underflow."""
    with np.errstate(over="ignore", under="ignore"):
        log = y if not sigmoid else np.where(y > 0, -np.log1p(np.exp(-np.abs(y))), y - np.log1p(np.exp(-np.abs(y))))
        e = np.exp(log - log.max())
    return e / e.sum()


def _first(values, count):
    """Indices of the `count` largest values above -inf, descending, ties to the lower index."""
    order = sorted(range(len(values)), key=lambda i: (-values[i], i))
    return [i for i in order[:count] if values[i] > -np.inf]


def route(x, k, sigmoid, bias=None, groups=1, keep=1, group_top=1, renorm=True, scale=1.0, mask=None):
    """-> (idx int32 [bs, k], weights float64 [bs, k], relative tolerance [bs, k] of a binary32 evaluation).

    The tolerance counts, per chosen score, one step of e^x (2 U), the rounded
    difference in its argument (|d| U), and for the sigmoid a sum and a
    quotient (2 U); for a sum the same of its terms and one rounding for each
    addition in a tree of at most 38; then the quotient and the scale (2 U)."""
    bs, e = x.shape
    idx = np.full((bs, k), -1, np.int32)
    w = np.zeros((bs, k))
    tol = np.zeros((bs, k))
    ok_all = eligible(x, mask)
    for t in range(bs):
        ok = ok_all[t]
        y = np.where(ok, np.minimum(np.where(ok, x[t], 0), np.finfo(np.float32).max), 0)
        s = scores(y, ok, sigmoid)
        u = np.where(ok, np.clip(np.rint((s + (0 if bias is None else bias)) * GRID) / GRID, -CLIP, CLIP), -np.inf)
        v = u if bias is not None else np.where(ok, y, -np.inf)
        if groups > 1:
            size = e // groups
            val = []
            for g in range(groups):
                part = np.sort((v if group_top == 1 else u)[g * size:(g + 1) * size])[::-1]
                part = part[part > -np.inf][:group_top]
                val.append(part.sum() if len(part) else -np.inf)
            kept = _first(val, keep)
            v = np.where(np.isin(np.arange(e) // size, kept), v, -np.inf)
        at = _first(v, k)
        if not at:
            continue
        idx[t, :len(at)] = at
        c = y[at]
        if renorm:
            w[t, :len(at)] = shares(c, sigmoid) * scale
            d = np.abs(c - min(c.max(), 0.0)) if sigmoid else c.max() - c
            d = np.minimum(d, 200.0)  # past that the score is 0 either way
            tol[t, :len(at)] = ((4 + d) + (4 + d.max()) + 38 + 2) * U
        else:
            w[t, :len(at)] = s[at] * scale
            d = np.minimum(np.abs(c) if sigmoid else y[ok].max() - c, 200.0)
            far = 0.0 if sigmoid else float((s[ok] * (y[ok].max() - y[ok])).sum())
            tol[t, :len(at)] = ((4 + d) + (4 + far) + 38 + 2) * U
    return idx, w, tol


def route_backward(g, x, idx, sigmoid, renorm=True, scale=1.0):
    """-> (dx float64 [bs, E], magnitude [bs, E]): the gradient, and the sum of
    the absolute terms that make each of its values up (what a rounding error
    in a term is relative to)."""
    bs, e = x.shape
    dx, mag = np.zeros((bs, e)), np.zeros((bs, e))
    ok_all = eligible(x)
    for t in range(bs):
        ok = ok_all[t]
        y = np.where(ok, np.minimum(np.where(ok, x[t], 0), np.finfo(np.float32).max), 0)
        js = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < e and ok[idx[t, j]]]
        if not js:
            continue
        at, gg = idx[t, js], g[t, js].astype(np.float64) * scale
        s = scores(y, ok, sigmoid)
        if renorm:
            a = shares(y[at], sigmoid)
            slope = scores(-y[at], np.ones(len(at), bool), True) if sigmoid else 1.0
            dx[t, at] = a * (gg - (gg * a).sum()) * slope
            mag[t, at] = a * (np.abs(gg) + (np.abs(gg) * a).sum()) * slope
        elif sigmoid:
            slope = scores(-y[at], np.ones(len(at), bool), True)
            dx[t, at] = gg * s[at] * slope
            mag[t, at] = np.abs(dx[t, at])
        else:
            ds = np.zeros(e)
            ds[at] = gg
            dx[t] = s * (ds - (ds * s).sum())
            mag[t] = s * (np.abs(ds) + (np.abs(ds) * s).sum())
    return dx, mag


def to_type(values, kind):
    """Rounded once to bf16, fp16 or fp32; returned as float32 values."""
    v = np.asarray(values, np.float32)
    if kind == "fp32":
        return v
    if kind == "fp16":
        with np.errstate(over="ignore"):
            return v.astype(np.float16).astype(np.float32)
    b = v.view(np.uint32)
    r = ((b + 0x7fff + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return np.where(np.isnan(v), v, r.view(np.float32))


HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
# absolute: half a step among the type's subnormal values
TINY = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}


def logits(rng, bs, e, kind, spread=1.5):
    return to_type(rng.standard_normal((bs, e)) * spread + rng.standard_normal((1, e)) * 0.5, kind)
