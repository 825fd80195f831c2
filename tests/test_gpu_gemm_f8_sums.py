"""The sums of the 8-bit float product: exact cases whose scales differ from
block to block, bit for bit; the error of normal rows as a whole; and outliers
that cancel, against the stated bound.  Every kernel, every type of result."""

import numpy as np
import pytest

import block_rows_ref as B
import f8_sums_ref as S
from gpu_util import log
from instance_cases_f8 import PLAIN, WIDE
from test_gpu_gemm_f8 import inputs, run_plain

pytestmark = pytest.mark.gpu

KERNELS = [(name, kind) for kind in ("bf16", "fp16", "fp32") for name in PLAIN]


def shape(name, kind):
    rows, n, counts = (WIDE if kind == "fp32" else PLAIN)[name]
    return rows, n, counts, B.owners(counts, rows)


def exact_kernel(name, kind):
    """Whether every product is kept."""
    return kind == "fp32" or name == "split16"


def of_type(want, kind):
    assert np.abs(want).max() < 65504
    return S.rounded(want, kind)


@pytest.mark.parametrize("name,kind", KERNELS)
@pytest.mark.parametrize("k", [144, 640, 1296, 4096])
def test_blocks_scaled_by_powers_of_two_bit_for_bit(name, kind, k):
    """Codes of -3 .. 3 (products of at most 9, which the 8-bit instruction keeps beside each other) and scales of 2^-2 ..
    2^2: a sum is a multiple of 2^-4, and below 2^20 at these k with terms of any sign, so binary32 holds it."""
    rows, n, counts, own = shape(name, kind)
    rng = np.random.default_rng(k)
    a, ts, w, ws = inputs(rng, rows, k, n, len(counts), 1, exact=True)
    ts, ws = 2.0 ** rng.integers(-2, 3, ts.shape), 2.0 ** rng.integers(-2, 3, ws.shape)
    log(f"gemm_f8 powers of two {name} {kind} {k}")
    got = run_plain(a, ts, w, ws, counts, kind)
    want, _ = B.product(a, ts, w, ws, own, n)
    assert B.blocks(k) * 128 * 9 * 16 < 2 ** 20
    assert np.array_equal(got[own >= 0], of_type(want[own >= 0], kind))


@pytest.mark.parametrize("name,kind", KERNELS)
def test_one_block_keeps_its_scales_whole(name, kind):
    """One block of k: its sum of at most 1152 has 11 bits, a row's scale 13 bits and a column's 1, so the result is
    rounded once and a scale that lost bits shows."""
    rows, n, counts, own = shape(name, kind)
    rng = np.random.default_rng(n)
    a, ts, w, ws = inputs(rng, rows, 128, n, len(counts), 1, exact=True)
    ts, ws = (4097 + 2 * rng.integers(0, 2048, ts.shape)) / 4096, 2.0 ** rng.integers(-2, 3, ws.shape)
    log(f"gemm_f8 one block {name} {kind}")
    got = run_plain(a, ts, w, ws, counts, kind)
    want, _ = B.product(a, ts, w, ws, own, n)
    assert np.array_equal(got[own >= 0], of_type(want[own >= 0], kind))


@pytest.mark.parametrize("name,kind", KERNELS)
@pytest.mark.parametrize("k", [272, 1152, 2064])
def test_normal_rows_as_a_whole(name, kind, k):
    rows, n, counts, own = shape(name, kind)
    a, ts, w, ws = inputs(np.random.default_rng(k), rows, k, n, len(counts), 1)
    log(f"gemm_f8 norm of the error {name} {kind} {k}")
    got = run_plain(a, ts, w, ws, counts, kind)
    want, _ = B.product(a, ts, w, ws, own, n)
    S.check_norm(got[own >= 0], want[own >= 0], kind, S.EXACT if exact_kernel(name, kind) else S.STATED)


@pytest.mark.parametrize("name,kind", KERNELS)
def test_outliers_that_cancel(name, kind):
    """Of each eight products two are 448 * 448 and its negative, the others below the largest's 2^-13 and above: what is
    left is theirs.  Products are multiples of 1/2 and a block's sums below 2^22, so binary32 holds every one on the way:
    where all products are kept, only the scales' roundings (a product, a multiply-add a block, and four parts' sums)
    are left.  Elsewhere the result is within what seven products below 2^-13 of the largest of each eight may be."""
    rows, n, counts, own = shape(name, kind)
    k = 400
    rng = np.random.default_rng(7)
    a, ts, w, ws = inputs(rng, rows, k, n, len(counts), 1)
    a = B.e4m3(rng.choice([0.0, 1.0, 2.0, 3.0, 8.0, 15.0], a.shape))
    w = B.e4m3(rng.choice([0.0, 1.0, 1.5, 2.0, 4.0], w.shape))
    plus = np.arange(k // 8) * 8 + rng.integers(0, 4, k // 8)
    minus = np.arange(k // 8) * 8 + rng.integers(4, 8, k // 8)
    a[:, plus] = a[:, minus] = 448
    w[:, :, plus], w[:, :, minus] = 448, -448
    log(f"gemm_f8 outliers that cancel {name} {kind}")
    got = run_plain(a, ts, w, ws, counts, kind)
    at = own >= 0
    want, err = B.product(a, ts, w, ws, own, n)
    if exact_kernel(name, kind):
        err = np.zeros_like(want)
        for b in range(B.blocks(k)):
            part = np.where(np.arange(k) // 128 == b, a, 0.0)
            err += (B.blocks(k) + 6) * B.U * np.abs(B.product(part, ts, w, ws, own, n)[0])
    else:
        err = err + B.cut(a, ts, w, ws, own, n)
    assert B.near(got[at], want[at], kind, err[at])
