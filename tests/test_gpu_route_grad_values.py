"""The router's gradient for weight gradients that are infinite or NaN: experts that are not eligible get 0 whatever the
gradients hold, and other tokens are not touched."""

import numpy as np
import pytest
import torch

import combine_moe_layout_03_amd as M
import router_ref as R
from gpu_util import log
from test_gpu_route import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs,e,k", [(9, 70, 5), (2053, 64, 6), (2050, 256, 8), (3, 1500, 20)])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan, 3e38], ids=str)
def test_ineligible_experts_get_zero(bs, e, k, sigmoid, renorm, value):
    rng = np.random.default_rng(e)
    x = R.logits(rng, bs, e, "fp32")
    idx = np.stack([rng.permutation(e)[:k] for _ in range(bs)]).astype(np.int32)
    off = np.zeros((bs, e), bool)
    off[:, rng.permutation(e)[: e // 4]] = True
    np.put_along_axis(off, idx[:, :1], False, axis=1)  # the first entry stays
    x[off] = np.where(rng.random(off.sum()) < 0.5, np.nan, -np.inf)
    g = rng.standard_normal((bs, k)).astype(np.float32)
    bad = np.arange(0, bs, 2)
    g[bad, 0] = value
    out = torch.full((bs, e), 9.0, device="cuda")
    log(f"route_backward {value} among the gradients {bs} {e} {k} sigmoid={sigmoid} renorm={renorm}")
    score = M.MOE_SCORE_SIGMOID if sigmoid else M.MOE_SCORE_SOFTMAX
    args = (dev(x), torch.from_numpy(idx).cuda(), score)
    M.moe_route_backward(dev(g), *args, out, renormalize=renorm, scale=2.0)
    clean = np.where(np.arange(bs)[:, None] % 2 == 0, 1.0, g).astype(np.float32)
    want = torch.full((bs, e), 9.0, device="cuda")
    M.moe_route_backward(dev(clean), *args, want, renormalize=renorm, scale=2.0)
    torch.cuda.synchronize()
    got, want = out.cpu().numpy(), want.cpu().numpy()
    assert (got[off] == 0).all()
    assert np.array_equal(got[1::2], want[1::2])
    assert not np.isfinite(got[bad, idx[bad, 0]]).any() or value == 3e38
