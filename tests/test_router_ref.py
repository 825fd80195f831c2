"""The 64-bit definitions that the GPU tests compare with: the gradients'
formulas against central differences, and the router's choice against a
direct enumeration (CPU only)."""

import itertools

import numpy as np
import pytest

import router_ref as R


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_matches_differences(sigmoid, renorm):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 10))
    x[1, 3] = -np.inf
    idx, _, _ = R.route(x, 3, sigmoid, renorm=renorm)
    g = rng.standard_normal((4, 3))
    dx, _ = R.route_backward(g, x, idx, sigmoid, renorm, 1.7)

    def loss(z):
        total = 0.0
        for t in range(4):
            ok = R.eligible(z)[t]
            s = R.scores(np.where(ok, z[t], 0), ok, sigmoid)[idx[t]]
            total += (g[t] * 1.7 * (s / s.sum() if renorm else s)).sum()
        return total

    h = 1e-5
    for t, e in itertools.product(range(4), range(10)):
        if x[t, e] == -np.inf:
            assert dx[t, e] == 0
            continue
        up, down = x.copy(), x.copy()
        up[t, e] += h
        down[t, e] -= h
        # central differences: h^2 f''' / 6 and a rounding of f over h, both below 1e-8 here
        assert abs((loss(up) - loss(down)) / (2 * h) - dx[t, e]) < 1e-8


def test_route_choice_against_enumeration():
    rng = np.random.default_rng(4)
    for case in range(40):
        x = np.round(rng.standard_normal((1, 8)) * 2) / 2  # many ties
        bias = np.round(rng.standard_normal(8)) / 4
        idx, w, _ = R.route(x, 3, True, bias=bias, groups=4, keep=2, group_top=2, scale=2.0)
        s = 1 / (1 + np.exp(-x[0]))
        u = s + bias
        best = max(itertools.combinations(range(4), 2), key=lambda p: (
            sorted((round(u[2 * g] + u[2 * g + 1], 8) for g in p), reverse=True), [-g for g in p]))
        members = [e for e in range(8) if e // 2 in best]
        want = sorted(members, key=lambda e: (-round(u[e], 8), e))[:3]
        assert list(idx[0]) == want
        assert np.allclose(w[0], 2.0 * s[want] / s[want].sum(), rtol=1e-12)


def test_rows_without_experts():
    x = np.array([[np.nan, -np.inf, -np.inf], [0.0, np.nan, -np.inf]])
    idx, w, _ = R.route(x, 2, False, mask=np.array([1, 1]))
    assert idx.tolist() == [[-1, -1], [0, -1]] and w.tolist() == [[0, 0], [1, 0]]
    dx, _ = R.route_backward(np.ones((2, 2)), x, idx, False)
    assert not dx.any()
