"""The router's choice where scores are small, close or negative with their bias, against the choice by 80-bit scores
(router_choice_ref.py) and without a grid."""

import numpy as np
import pytest

import router_choice_ref as C
import router_ref as R
from gpu_util import log
from test_gpu_route import run_route
from test_router_choice_ref import FAR

pytestmark = pytest.mark.gpu
# Two exponentials and a sum put a softmax score off by less than 2^-40 of itself, and values keep 42 bits: unequal
# values further apart than this (relative to the larger) are told apart.  A row in which two are closer is left out.
GAP = 2.0 ** -38

# bs, E, k, groups, keep: a wave and 16 lanes a token; groups of whole lanes, parts of lanes and neither
SHAPES = [(40, 64, 6, 8, 3), (30, 60, 4, 5, 2), (20, 256, 8, 8, 4), (12, 352, 9, 2, 1), (6, 1000, 10, 10, 4), (24, 2048, 16, 64, 8),
          (2050, 16, 4, 4, 2), (2049, 30, 3, 5, 2), (2100, 64, 6, 8, 3), (2048, 160, 6, 8, 3), (2051, 256, 8, 8, 4)]


def check(x, kind, k, sigmoid, bias=None, rows=None, **kw):
    """The call on all rows; the reference on `rows` of them (the others repeat them)."""
    idx, w = run_route(x, kind, k, sigmoid, bias, **kw)
    rows = rows or len(x)
    want, gap = C.choose(x[:rows].astype(np.float64), k, sigmoid, None if bias is None else bias.astype(np.float64), **kw)
    clear = gap > GAP
    assert clear.mean() > 0.5, gap  # the inputs' own property
    want, clear = (np.concatenate([v] * -(-len(x) // rows))[:len(x)] for v in (want, clear))
    assert np.array_equal(idx[clear], want[clear]), np.argwhere((idx != want) & clear[:, None])[:5]
    assert np.isfinite(w).all()


def repeated(rng, bs, e, make):
    """Logits of at most 100 different rows, repeated to bs."""
    rows = min(bs, 100)
    return np.tile(make(rows), (-(-bs // rows), 1))[:bs], rows


@pytest.mark.parametrize("row", FAR, ids=lambda r: str(r[0]))
@pytest.mark.parametrize("bs", [1, 2048])
def test_scores_far_below_one(row, bs):
    x = np.tile(np.array([row[0]], np.float32), (bs, 1))
    log(f"route far scores {row} {bs}")
    idx, _ = run_route(x, "fp32", row[3], row[1], groups=4, keep=row[2], group_top=2)
    assert (idx == row[4]).all()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_groups_of_small_scores(shape, kind):
    """Groups ranked by sums of two scores, softmax logits up to some 300 below the top, sigmoid logits of -10 to -104."""
    bs, e, k, groups, keep = shape
    rng = np.random.default_rng(e + bs)
    x, rows = repeated(rng, bs, e, lambda n: R.logits(rng, n, e, kind, spread=40))
    log(f"route small scores {shape} {kind} softmax")
    check(x, kind, k, False, rows=rows, groups=groups, keep=keep, group_top=2)
    y, rows = repeated(rng, bs, e, lambda n: R.to_type(rng.uniform(-104, -10, (n, e)), kind))
    log(f"route small scores {shape} {kind} sigmoid")
    check(y, kind, k, True, rows=rows, groups=groups, keep=keep, group_top=2)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_biases_of_every_size(shape, sigmoid):
    """Zeros, and biases from 2^-100 to 1, beside scores as small."""
    bs, e, k, groups, keep = shape
    rng = np.random.default_rng(e * bs)
    for bias in (np.zeros(e, np.float32), np.exp2(rng.uniform(-100, 0, e)).astype(np.float32)):
        x, rows = repeated(rng, bs, e, lambda n: R.to_type(
            rng.uniform(-100, 10, (n, e)) if sigmoid else rng.standard_normal((n, e)) * 30, "fp32"))
        for top in (1, 2):
            log(f"route biases of every size {shape} sigmoid={sigmoid} top={top}")
            check(x, "fp32", k, sigmoid, bias, rows, groups=groups, keep=keep, group_top=top)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_negative_values_and_ties(shape, sigmoid):
    """Scores below their bias: negative values, many of them equal, of which the lower id comes first."""
    bs, e, k, groups, keep = shape
    rng = np.random.default_rng(3 * e + bs)
    bias = (-2.0 - rng.integers(0, 3, e) / 4).astype(np.float32)
    x, rows = repeated(rng, bs, e, lambda n: np.round(rng.standard_normal((n, e))).astype(np.float32))
    x[0] = x[rows % len(x)] = 0.0
    x = np.tile(x[:rows], (-(-bs // rows), 1))[:bs]
    for top in (1, 2):
        log(f"route negative values {shape} sigmoid={sigmoid} top={top}")
        check(x, "fp32", k, sigmoid, bias, rows, groups=groups, keep=keep, group_top=top)
    log(f"route equal negative values {shape} sigmoid={sigmoid}")
    idx, _ = run_route(np.zeros_like(x), "fp32", k, sigmoid, np.full(e, -3.0, np.float32))
    assert (idx == np.arange(k)).all()


def test_values_of_zero():
    """A score that its bias cancels stands between the positive and the negative values, ties to the lower id."""
    x = np.zeros((3, 40), np.float32)
    bias = np.full(40, -0.5, np.float32)
    x[:, 5], x[:, 30], x[:, 0], x[:, 8] = 0.25, 0.5, -0.25, -0.5
    log("route values of zero")
    idx, _ = run_route(x, "fp32", 32, True, bias)
    zero = [e for e in range(40) if e not in (0, 5, 8, 30)]
    assert (idx == ([30, 5] + zero)[:32]).all()
    idx, _ = run_route(x[:, :12].copy(), "fp32", 12, True, bias[:12])
    assert (idx == [5, 1, 2, 3, 4, 6, 7, 9, 10, 11, 0, 8]).all()


def test_logits_at_the_type_limits():
    """Without a bias the logits themselves are compared, up to the largest and smallest of the type."""
    big = np.finfo(np.float32).max
    x = np.array([[-big, big, 0.0, -1e-45, 1e-45, -np.inf, 1.0, -1.0, np.nextafter(np.float32(1), np.float32(2)), -0.0, 1e38,
                   -1e38]], np.float32)
    log("route logits at the limits")
    idx, _ = run_route(x, "fp32", 12, True)
    assert idx[0].tolist() == [1, 10, 8, 6, 4, 2, 9, 3, 7, 11, 0, -1]
