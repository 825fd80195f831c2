"""Biases that are not finite: an expert whose bias is -inf or NaN is not chosen, counts for no group, and keeps its
place in the softmax's sum; +inf counts as the largest value."""

import numpy as np
import pytest

import router_ref as R
from gpu_util import log
from test_gpu_route import run_route

pytestmark = pytest.mark.gpu


def expected(x, k, sigmoid, bias, groups, keep, top):
    """The choice with the experts of a bias of -inf or NaN taken out by hand, and the scores of the others from the
    whole row."""
    out = ~(bias > -np.inf)
    finite = np.where(out, 0, np.minimum(bias, 1e6))
    idx = np.full((len(x), k), -1)
    w = np.zeros((len(x), k))
    for t, row in enumerate(x.astype(np.float64)):
        ok = R.eligible(row[None])[0]
        s = R.scores(np.where(ok, row, 0), ok, sigmoid)
        u = np.where(ok & ~out, np.clip(s + finite, -R.CLIP, R.CLIP), -np.inf)
        size = len(u) // groups
        val = []
        for g in range(groups):
            part = np.sort(u[g * size:(g + 1) * size])[::-1][:top]
            part = part[part > -np.inf]
            val.append(part.sum() if len(part) else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-val[g], g))[:keep]
        v = np.where(np.isin(np.arange(len(u)) // size, kept), u, -np.inf)
        at = [e for e in sorted(range(len(u)), key=lambda e: (-v[e], e))[:k] if v[e] > -np.inf]
        idx[t, :len(at)] = at
        w[t, :len(at)] = s[at]
    return idx, w


# bs, E, k, groups, keep, group_top: a wave and 16 lanes a token, groups of whole lanes and not, several widths of lane
@pytest.mark.parametrize("shape", [(7, 64, 6, 1, 1, 1), (9, 60, 9, 5, 3, 2), (5, 256, 8, 8, 4, 2), (3, 1000, 10, 10, 4, 1),
                                   (2049, 160, 6, 8, 3, 2), (2050, 16, 4, 4, 2, 1), (2048, 256, 9, 8, 8, 1),
                                   (2051, 256, 8, 8, 4, 2)], ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("values", [[np.nan], [-np.inf], [np.nan, -np.inf]], ids=["nan", "inf", "both"])
def test_experts_switched_off(shape, sigmoid, values):
    bs, e, k, groups, keep, top = shape
    rng = np.random.default_rng(e + k)
    x = R.logits(rng, bs, e, "fp32")
    bias = (rng.standard_normal(e) * 0.05).astype(np.float32)
    off = rng.permutation(e)[: e // 3]
    bias[off] = np.resize(values, len(off))
    x[0, off] = 30.0  # the largest logits of all would be chosen first
    log(f"route bias switched off {shape} {values} sigmoid={sigmoid}")
    idx, w = run_route(x, "fp32", k, sigmoid, bias, groups=groups, keep=keep, group_top=top, renorm=False)
    want, ww = expected(x, k, sigmoid, bias, groups, keep, top)
    assert np.array_equal(idx, want), np.argwhere(idx != want)[:5]
    assert not np.isin(idx, off).any()
    for row in idx:
        row = row[row >= 0]
        assert len(set(row)) == len(row)
    # a score takes a difference, an exponential, a sum of at most 38 additions in a tree, and a quotient, in binary32;
    # the exponent's rounding is relative to its size
    assert (np.abs(w - ww) <= (2 * (4 + 64) + 40) * R.U * ww).all()


def test_every_expert_switched_off_or_few_left():
    rng = np.random.default_rng(4)
    x = R.logits(rng, 5, 32, "fp32")
    for left in (0, 1, 3):
        bias = np.full(32, -np.inf, np.float32)
        bias[::3] = np.nan
        bias[7:7 + left] = 0.25
        log(f"route bias: {left} experts left")
        for groups, keep, top in ((1, 1, 1), (4, 2, 2), (4, 2, 1)):
            idx, w = run_route(x, "fp32", 8, True, bias, groups=groups, keep=keep, group_top=top)
            want, _ = expected(x, 8, True, bias, groups, keep, top)
            assert np.array_equal(idx, want) and (w[idx < 0] == 0).all() and np.isfinite(w).all()


def test_infinite_bias_is_the_largest():
    x = R.logits(np.random.default_rng(5), 6, 40, "fp32")
    bias = np.zeros(40, np.float32)
    bias[[4, 11]] = np.inf
    bias[20] = 1e30
    log("route bias: infinite")
    idx, w = run_route(x, "fp32", 5, False, bias)
    assert (idx[:, :3] == [4, 11, 20]).all() and np.isfinite(w).all()
