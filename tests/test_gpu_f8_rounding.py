"""The rounding to 8 and 16 bits, bit for bit: every e4m3 value, the middles
between neighbours and the floats beside them, in blocks whose largest magnitude
is 448, so that scale and factor are 1 and nothing else is rounded."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log
from instance_cases_f8 import GATED
from test_gpu_gemm_f8 import run_gated

pytestmark = pytest.mark.gpu


def e4m3_values():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    return np.unique(every[np.isfinite(every)])  # (one zero)


def near_middles():
    every = e4m3_values()
    mid = ((every[1:] + every[:-1]) / 2).astype(np.float32)
    return np.concatenate([every.astype(np.float32), mid, np.nextafter(mid, np.float32(500)),
                           np.nextafter(mid, np.float32(-500))])


def test_the_values_tell_roundings_apart():
    """Half-even is the only one of the usual roundings that gives what the tests below ask for."""
    every = e4m3_values()
    mid = (every[1:] + every[:-1]) / 2
    want = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy()
    away = np.where(mid > 0, every[1:], every[:-1])
    to_zero = np.where(mid > 0, every[:-1], every[1:])
    assert np.array_equal(want, B.e4m3(mid))
    assert all((want != other).sum() > 100 for other in (every[1:], every[:-1], away, to_zero))


@pytest.mark.parametrize("hidden", [128, 512, 1152, 4096, 8192, 16384])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_norm_rounds_half_even(hidden, kind):
    """Rows of ones and eps 0: rstd is 1 and y is the weight."""
    values, rng = near_middles(), np.random.default_rng(hidden)
    x = torch.ones((3, hidden), dtype=B.TYPES[kind], device="cuda")
    blocks = hidden // 128
    for part in range(-(-values.size // (127 * blocks))):
        w = np.resize(np.roll(values, -part * 127 * blocks), (blocks, 127))
        w = np.concatenate([w, np.full((blocks, 1), 448, np.float32)], axis=1)
        w = rng.permuted(w, axis=1).reshape(-1)
        weight = torch.from_numpy(w)
        for out_kind in ("bf16", "fp16", "fp32"):
            rows = torch.full((3 * B.row_bytes(hidden),), 0xA5, dtype=torch.uint8, device="cuda")
            out, rstd = torch.zeros((3, hidden), dtype=B.TYPES[out_kind], device="cuda"), torch.zeros(3, device="cuda")
            log(f"rms_norm rounding {hidden} {kind} {out_kind} part {part}")
            M.moe_rms_norm(x, weight.cuda(), 0.0, out=out, rows=rows, rstd=rstd)
            torch.cuda.synchronize()
            codes, scales = B.unpack(rows, 3, hidden)
            assert (rstd == 1).all() and (scales == 1).all()
            want = weight.to(torch.float8_e4m3fn).double().numpy()
            assert all(np.array_equal(c, want) for c in codes)
            assert all(torch.equal(o, weight.to(B.TYPES[out_kind])) for o in out.cpu())


@pytest.mark.parametrize("name", GATED)
def test_gated_product_rounds_half_even(name):
    """A gate of 128, whose e^-128 is below binary32, and up columns of a value and half a step: the activation is the
    middle between two codes."""
    rows, n, counts = GATED[name]
    every = e4m3_values()
    low, step = every[:-1], np.diff(every)
    at = np.resize(np.random.default_rng(0).permutation(low.size), n)
    value, half = low[at], step[at] * 8  # (times 2^-4)
    value[::128], half[::128] = 448, 0
    k, groups = 32, len(counts)
    a, w = np.zeros((rows, k)), np.zeros((groups, 2 * n, k))
    a[:, 0], a[:, 17] = 1, 2.0 ** -4
    w[:, :n, 0] = 128
    w[:, n:, 0], w[:, n:, 17] = value, half
    assert np.array_equal(B.e4m3(w), w)
    ws = np.ones((groups, 2 * B.blocks(n), 1))
    ws[:, B.blocks(n):] = 2.0 ** -7
    log(f"gemm_swiglu_f8 rounding {name}")
    out = run_gated(a, np.ones((rows, 1)), w, ws, counts)
    own = B.owners(counts, rows) >= 0
    codes, scales = B.unpack(out, rows, n)
    assert (scales[own] == 1).all()
    assert (codes[own] == B.e4m3(value + half / 16)).all()
