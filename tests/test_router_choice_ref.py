"""The choice by ungridded scores (CPU only): hand-worked rows, agreement with a grid of 2^-30 where scores are large, and
the rows in which such a grid loses their order."""

import numpy as np
import pytest

import router_choice_ref as C
import router_ref as R

# logits, score, groups kept of 4, entries, the experts that the scores choose; group values are sums of two scores
FAR = [
    ([30, 29, 0, 0, 5, 5, 4, 4], False, 2, 4, [0, 1, 4, 5]),
    ([-30, -29, -40, -40, -23, -23, -24, -24], True, 1, 2, [4, 5]),
    ([200, 199, 0, 0, 1, 1, 0, 0.5], False, 2, 4, [0, 1, 4, 5]),
    ([0, 0, 400, -200, -90, -190, -100, -100], False, 2, 3, [2, 0, 1]),
    ([-100, -101, -103, -90, -95, -91, -200, -300], True, 2, 4, [3, 5, 4, 2]),
]


@pytest.mark.parametrize("row", FAR, ids=lambda r: str(r[0]))
def test_scores_far_below_one(row):
    x, sigmoid, keep, k, want = np.array([row[0]], np.float64), row[1], row[2], row[3], row[4]
    got, gap = C.choose(x, k, sigmoid, groups=4, keep=keep, group_top=2)
    assert got[0].tolist() == want and gap[0] > 1e-3


def test_the_grid_loses_their_order():
    lost = [R.route(np.array([row[0]], np.float64), row[3], row[1], groups=4, keep=row[2], group_top=2)[0][0].tolist()
            != row[4] for row in FAR]
    assert sum(lost) >= 3


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_agrees_with_the_grid_on_large_scores(sigmoid, biased):
    rng = np.random.default_rng(1)
    x = R.logits(rng, 60, 64, "fp32").astype(np.float64)
    x[3, ::2], x[4, 5:], x[5, 7], x[6] = np.nan, -np.inf, np.inf, 0.0
    bias = rng.standard_normal(64) * 0.05 if biased else None
    for groups, keep, top in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
        want = R.route(x, 6, sigmoid, bias, groups, keep, top)[0]
        got, gap = C.choose(x, 6, sigmoid, bias, groups, keep, top)
        assert gap.min() > 2.0 ** -30 and np.array_equal(got, want)


def test_softmax_of_wide_logits_with_a_bias_of_zeros():
    """A grid of 2^-30 chooses other experts for about one token in a hundred."""
    x = R.logits(np.random.default_rng(2), 400, 256, "fp32", spread=10).astype(np.float64)
    none, _ = C.choose(x, 8, False)
    zeros, gap = C.choose(x, 8, False, np.zeros(256))
    assert gap.min() > 2.0 ** -40 and np.array_equal(none, zeros)
    grid = R.route(x, 8, False, np.zeros(256))[0]
    assert 0 < (grid != none).any(axis=1).sum() < 20


def test_values_are_cut():
    v = np.array([1.0, -1.0, 1 + 2.0 ** -41, 1 + 2.0 ** -42, -1 - 2.0 ** -42, 3e-300, 0.0, -np.inf, np.pi], np.longdouble)
    got = C.cut(v)
    assert (got[:3] == v[:3]).all() and got[3] == 1 and got[4] == -1 and got[6] == 0 and got[7] == -np.inf
    assert 0 <= (v[5] - got[5]) / v[5] < 2.0 ** -41 and 0 < np.pi - got[8] < 2.0 ** -40
