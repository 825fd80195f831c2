"""The check of the 8-bit float products' sums sees what the bound of single results lets pass (CPU)."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import f8_sums_ref as S


def case(k, seed=0, rows=64, n=256):
    """Codes, scales, and the products of one expert in 64 bits."""
    rng = np.random.default_rng(seed)
    a, w = (B.e4m3(np.clip(rng.normal(size=s) * 120, -448, 448)) for s in ((rows, k), (1, n, k)))
    ts = ((rng.random((rows, B.blocks(k))) + 0.2) / 100).astype(np.float32).astype(np.float64)
    ws = ((rng.random((1, B.blocks(n), B.blocks(k))) + 0.2) / 100 / np.sqrt(k)).astype(np.float32).astype(np.float64)
    return a, ts, w, ws


def product(a, ts, w, ws):
    return B.product(a, ts, w, ws, np.zeros(a.shape[0], int), w.shape[1])[0]


def refused(got, want, kind, off):
    try:
        S.check_norm(got, want, kind, off)
    except AssertionError:
        return True
    return False


def to_bf16(v):
    return torch.from_numpy(v).bfloat16().double().numpy()


@pytest.mark.parametrize("k", [256, 1152, 2064])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_right_results_pass(k, kind):
    """Rounded once, and summed by binary32 in blocks (torch on the host)."""
    a, ts, w, ws = case(k)
    want = product(a, ts, w, ws)
    S.check_norm(S.rounded(want, kind), want, kind, 0.0)
    f = torch.from_numpy
    full = f(a).float() * f(B.spread(ts, k)).float()
    other = f(w[0]).float() * f(np.repeat(B.spread(ws[0], k), 128, axis=0)).float()
    S.check_norm((full @ other.t()).to(B.TYPES[kind]).double().numpy(), want, kind, S.EXACT)


@pytest.mark.parametrize("k", [256, 1152, 2064])
@pytest.mark.parametrize("spoil", ["scales in bf16", "weight scales in bf16", "a scale of 1.004", "a term left out",
                                   "a block's scale of its neighbour", "sums in fp16"])
def test_wrong_results_are_refused(k, spoil):
    a, ts, w, ws = case(k)
    want = product(a, ts, w, ws)
    if spoil == "scales in bf16":
        got = product(a, to_bf16(ts), w, ws)
    elif spoil == "weight scales in bf16":
        got = product(a, ts, w, to_bf16(ws))
    elif spoil == "a scale of 1.004":
        got = want * 1.004
    elif spoil == "a term left out":
        b = a.copy()
        b[:, k // 2] = 0
        got = product(b, ts, w, ws)
    elif spoil == "a block's scale of its neighbour":
        t = ts.copy()
        t[:, 0] = ts[:, 1]
        got = product(a, t, w, ws)
    else:
        got = sum(S.rounded(product(np.where(np.arange(k) // 128 == b, a, 0), ts, w, ws), "fp16")
                  for b in range(B.blocks(k)))
    assert refused(S.rounded(got, "fp16"), want, "fp16", S.STATED)
    if spoil in ("scales in bf16", "weight scales in bf16") and k > 1000:  # the bound of single results lets these pass
        off = B.cut(a, ts, w, ws, np.zeros(a.shape[0], int), w.shape[1])
        assert B.near(S.rounded(got, "fp16"), want, "fp16", off)
    if spoil not in ("scales in bf16", "weight scales in bf16", "sums in fp16"):  # (less than bf16's own rounding)
        assert refused(S.rounded(got, "bf16"), want, "bf16", S.STATED)
