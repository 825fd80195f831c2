"""The norm's mean against a bound that counts the additions of a row of its width."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log

pytestmark = pytest.mark.gpu


def roundings(h):
    """Of 1 / sqrt(sum / h + eps): a lane's multiply-adds (8 for each of its 1, 2 or 4 chunks), the additions over 64
    lanes and over the row's waves (at most 8), the division and eps count half under the root; the root and the
    reciprocal follow."""
    chunks = 1 if h <= 512 else 2 if h <= 8192 else 4
    waves = -(-h // (512 * chunks))
    assert waves <= 8
    return (8 * chunks + 6 + waves - 1 + 2) / 2 + 2


@pytest.mark.parametrize("h", [8, 512, 520, 1024, 2048, 4104, 7168, 8192, 8200, 16384])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_rstd_to_its_own_roundings(h, kind):
    rng = np.random.default_rng(h)
    bs = 64
    x = torch.from_numpy(rng.normal(size=(bs, h)) * np.exp(rng.normal(size=(bs, 1)))).to(B.TYPES[kind]).cuda()
    w = torch.from_numpy((rng.random(h) + 0.5).astype(np.float32)).cuda()
    out, rstd = torch.zeros((bs, h), device="cuda"), torch.zeros(bs, device="cuda")
    log(f"rms_norm rstd {h} {kind}")
    M.moe_rms_norm(x, w, 1e-6, out=out, rstd=rstd)
    torch.cuda.synchronize()
    y, want = B.norm(x.cpu().double().numpy(), w.cpu().double().numpy(), float(np.float32(1e-6)))
    off = roundings(h) * B.U * 1.0001  # (products of roundings)
    assert off < 26 * B.U
    assert (np.abs(rstd.cpu().double().numpy() - want) <= off * want).all()
    assert (np.abs(out.cpu().double().numpy() - y) <= (off + 2.0001 * B.U) * np.abs(y)).all()
