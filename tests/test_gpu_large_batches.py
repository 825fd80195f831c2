"""Batches past one launch's threads: the router, its gradient and the combine's gradient on more than 2^26 tokens, whose
rows repeat a small table, against the same call on the table."""

import pytest
import torch

import combine_moe_layout_03_amd as M
from gpu_util import log

pytestmark = pytest.mark.gpu
BS = 2 ** 26 + 37
TABLE = 1009  # a prime, so that every part starts at another row of the table


def repeated(table):
    return table.repeat(-(-BS // TABLE), *([1] * (table.dim() - 1)))[:BS].contiguous()


def matches(got, table):
    """Whether got repeats the table (whole repeats as a view, then the rest)."""
    whole = BS // TABLE
    return bool((got[: whole * TABLE].view(whole, *table.shape) == table).all()) and torch.equal(
        got[whole * TABLE:], table[: BS - whole * TABLE])


@pytest.mark.parametrize("e,k,kind", [(17, 17, torch.bfloat16), (2, 1, torch.float32)])  # a wave, and 16 lanes, a token
def test_router(e, k, kind):
    gen = torch.Generator(device="cuda").manual_seed(e)
    table = (torch.randn((TABLE, e), device="cuda", generator=gen) * 2).to(kind)
    mask = (torch.rand((TABLE,), device="cuda", generator=gen) > 0.1).to(torch.uint8)

    def call(x, m):
        idx = torch.full((x.shape[0], k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((x.shape[0], k), float("nan"), device="cuda")
        M.moe_route(x, idx, w, M.MOE_SCORE_SIGMOID, renormalize=False, token_mask=m)
        return idx, w

    log(f"router: {BS} tokens, {e} experts")
    want_idx, want_w = call(table, mask)
    x = repeated(table)
    idx, w = call(x, repeated(mask))
    torch.cuda.synchronize()
    assert matches(idx, want_idx) and matches(w, want_w)
    log(f"router's gradient: {BS} tokens, {e} experts")
    g = torch.randn((TABLE, k), device="cuda", generator=gen)
    want = torch.full_like(table, 9.0)
    M.moe_route_backward(g, table, want_idx, M.MOE_SCORE_SIGMOID, want, renormalize=False)
    got = torch.full_like(x, 9.0)
    M.moe_route_backward(repeated(g), x, idx, M.MOE_SCORE_SIGMOID, got, renormalize=False)
    torch.cuda.synchronize()
    assert matches(got, want)


def test_combine_backward():
    """One expert and one entry a token, so that token t's row is row t."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    y, g = (torch.randn((TABLE, 8), device="cuda", generator=gen).bfloat16() for _ in range(2))
    w = torch.rand((TABLE, 1), device="cuda", generator=gen)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(yy, gg, ww):
        n = yy.shape[0]
        gr, gw = torch.full_like(yy, 9.0), torch.full_like(ww, 9.0)
        slot = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
        M.moe_combine_backward(gg, yy, M.MOE_BF16, torch.zeros_like(slot), ww, slot, zero, zero, 1, 1, gr, gw)
        return gr, gw

    log(f"combine_backward: {BS} entries")
    want = call(y, g, w)
    got = call(repeated(y), repeated(g), repeated(w))
    torch.cuda.synchronize()
    assert matches(got[0], want[0]) and matches(got[1], want[1])
