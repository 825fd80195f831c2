"""Batches of the norm past the rows of one launch."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log

pytestmark = pytest.mark.gpu

LAUNCH = 2 ** 21  # rows of one launch


@pytest.mark.parametrize("kind,out_kind", [("bf16", "fp32"), ("fp32", "fp16")])
def test_norm_of_several_launches(kind, out_kind):
    """Every output of a batch of two full launches and a few rows more is that of its parts called by themselves, bit for
    bit, and the rows on both sides of the borders are those of the definition."""
    bs, h, guard = 2 * LAUNCH + 5, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, residual = (torch.randn((bs, h), device="cuda", generator=gen).to(B.TYPES[kind]) for _ in range(2))
    weight = torch.rand(h, device="cuda", generator=gen) + 0.5

    def buffers(n):
        return (torch.full((n, h), 7, dtype=B.TYPES[kind], device="cuda"),
                torch.full((n, h), 7, dtype=B.TYPES[out_kind], device="cuda"),
                torch.full((n, B.row_bytes(h)), 0xA5, dtype=torch.uint8, device="cuda"),
                torch.full((n,), 7.0, device="cuda"))

    def run(first, n, to):
        s, out, rows, rstd = (t[:n] for t in to)
        M.moe_rms_norm(x[first:first + n], weight, 1e-6, residual=residual[first:first + n], sum=s, out=out, rows=rows,
                       rstd=rstd)
        torch.cuda.synchronize()

    log(f"rms_norm of {bs} rows {kind}")
    whole = buffers(bs + guard)
    run(0, bs, whole)
    for first in range(0, bs, LAUNCH):
        n = min(LAUNCH, bs - first)
        part = buffers(n)
        log(f"rms_norm rows {first} to {first + n}")
        run(first, n, part)
        assert all(torch.equal(w[first:first + n], p) for w, p in zip(whole, part))
    untouched = buffers(guard)
    assert all(torch.equal(w[bs:], u) for w, u in zip(whole, untouched))
    some = sorted({r for at in (0, LAUNCH, 2 * LAUNCH, bs) for r in range(at - 3, at + 3) if 0 <= r < bs})
    s, out, rows, rstd = (w[some] for w in whole)
    assert torch.equal(s, (x[some].float() + residual[some].float()).to(x.dtype))

    def host(t):
        return t.float().cpu().double().numpy()

    y, want = B.norm(host(s), host(weight), 1e-6)
    assert B.near(host(out), y, out_kind, B.NORM * np.abs(y)) and (np.abs(host(rstd) - want) <= B.RSTD * want).all()
    B.check_rows(*B.unpack(rows.contiguous(), len(some), h), y, B.NORM * np.abs(y))
