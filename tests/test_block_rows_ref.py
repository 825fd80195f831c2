"""The 64-bit reference of the norm, its gradient and the 8-bit rows, against
torch's own conversion and against differences (CPU)."""

import numpy as np
import torch

import block_rows_ref as B


def test_e4m3_rounding_agrees_with_torch():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    every = np.sort(every[np.isfinite(every)])
    assert np.array_equal(B.e4m3(every), every)
    middle = (every[1:] + every[:-1]) / 2  # exact in binary32, so torch rounds once
    v = np.concatenate([middle, np.nextafter(middle.astype(np.float32), np.float32(500)),
                        np.nextafter(middle.astype(np.float32), np.float32(-500)),
                        np.random.default_rng(0).normal(0, 100, 10000).astype(np.float32)]).clip(-448, 448)
    assert np.array_equal(B.e4m3(v), torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy())


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    s, w, g = rng.normal(size=(5, 48)), rng.random(48) + 0.5, rng.normal(size=(5, 48))
    eps, step = 1e-3, 1e-5
    y, rstd = B.norm(s, w, eps)
    dx, _, dw, _ = B.norm_backward(g, s, w, rstd)
    for _ in range(4):
        d, e = rng.normal(size=s.shape), rng.normal(size=48)
        up, down = B.norm(s + step * d, w, eps)[0], B.norm(s - step * d, w, eps)[0]
        assert abs(((up - down) * g).sum() / (2 * step) - (dx * d).sum()) < 1e-7
        up, down = B.norm(s, w + step * e, eps)[0], B.norm(s, w - step * e, eps)[0]
        assert abs(((up - down) * g).sum() / (2 * step) - (dw * e).sum()) < 1e-7


def test_rows_check_sees_a_wrong_code_and_scale():
    """The check that the GPU tests use refuses a code one step off, and a scale 2^-20 off."""
    rng = np.random.default_rng(2)
    y = rng.normal(size=(3, 272))
    d = np.maximum(B.block_max(y), B.TINY)
    codes, scales = B.e4m3(y * B.spread(448 / d, 272)), d / 448
    B.check_rows(codes, scales, y, 0.0 * y)
    for spoil in ("code", "scale"):
        c, s = codes.copy(), scales.copy()
        if spoil == "code":
            c[1, 200] = c[1, 200] * 1.125 if abs(c[1, 200]) < 400 else c[1, 200] * 0.875
        else:
            s[2, 1] *= 1 + 2.0 ** -20
        try:
            B.check_rows(c, s, y, 0.0 * y)
        except AssertionError:
            continue
        raise RuntimeError(spoil)
