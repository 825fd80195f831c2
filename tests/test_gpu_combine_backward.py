"""The combine's gradient: the rows' gradients bit for bit, the weights'
within the roundings of a binary32 sum, and both against differences of the
forward call."""

import numpy as np
import pytest
import torch

import combine_moe_layout_03_amd as M
import router_ref as R
from gpu_util import log

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FILL = 7.0  # in rows that no entry owns


def routes(rng, bs, k, epr, ranks, bad=0.1):
    """Ids with bad ones among them, their slots, offsets and bases, and each entry's row (-1: none)."""
    e = epr * ranks
    idx = rng.integers(0, e, (bs, k)).astype(np.int32)
    idx[rng.random((bs, k)) < bad] = -1
    idx[rng.random((bs, k)) < bad / 2] = e
    flat = idx.reshape(-1)
    ok = (flat >= 0) & (flat < e)
    count = np.bincount(flat[ok], minlength=e)
    start = np.cumsum(count) - count
    slot = np.full(flat.shape, -1, np.int32)
    seen = np.zeros(e, np.int64)
    row = np.full(flat.shape, -1, np.int64)
    for i in np.nonzero(ok)[0]:
        slot[i] = seen[flat[i]]
        seen[flat[i]] += 1
        row[i] = start[flat[i]] + slot[i]
    base = start[::epr].astype(np.int32)
    put = (start - np.repeat(start[::epr], epr)).astype(np.int32)
    return idx, slot.reshape(bs, k), put, base, row.reshape(bs, k)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def dev(x, kind):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(TYPES[kind])


def expected(g, y, w, row, kind, rows):
    """Row gradients [rows, h] as float32 (FILL where no entry's), weight gradients in 64 bits and their bounds."""
    bs, k = row.shape
    h = g.shape[1]
    out = np.full((rows, h), FILL, np.float32)
    dot, bound = np.zeros((bs, k)), np.zeros((bs, k))
    for t in range(bs):
        for j in range(k):
            if row[t, j] >= 0:
                out[row[t, j]] = R.to_type(w[t, j] * g[t], kind)
                prod = y[row[t, j]].astype(np.float64) * g[t]
                dot[t, j] = prod.sum()
                # 64 lanes or more share a row: so many additions in turn, then a tree of lanes and waves
                bound[t, j] = (8 * -(-h // 512) + 16) * R.U * np.abs(prod).sum()
    return out, dot, bound


@pytest.mark.parametrize("bs,h,k,epr,ranks", [(1, 8, 1, 1, 1), (3, 64, 4, 2, 3), (17, 1000, 5, 8, 3), (40, 2048, 8, 16, 2),
                                              (5, 7168, 8, 16, 16), (7, 4104, 9, 3, 2), (4, 520, 32, 40, 1),
                                              (2, 16384, 3, 4, 1), (6, 512, 17, 5, 4), (301, 72, 9, 6, 2),
                                              (131, 504, 5, 3, 4), (50, 520, 9, 7, 2)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("grad", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inplace", [False, True], ids=["", "inplace"])
def test_combine_backward(bs, h, k, epr, ranks, kind, grad, inplace):
    rng = np.random.default_rng(bs + h + k)
    idx, slot, put, base, row = routes(rng, bs, k, epr, ranks)
    g = R.to_type(rng.standard_normal((bs, h)), grad)
    y = R.to_type(rng.standard_normal((bs * k, h)), kind)
    y[np.setdiff1d(np.arange(bs * k), row[row >= 0])] = FILL
    w = rng.random((bs, k)).astype(np.float32)
    recv = dev(y, kind)
    out = recv if inplace else torch.full_like(recv, FILL)
    gw = torch.full((bs, k), float("nan"), device="cuda")
    log(f"combine_backward {bs} {h} {k} {epr}x{ranks} {kind} grad {grad} inplace={inplace}")
    M.moe_combine_backward(dev(g, grad), recv, M.dtype_code(TYPES[kind]), i32(idx), dev(w, "fp32"), i32(slot), i32(put),
                           i32(base), epr, ranks, out, gw)
    torch.cuda.synchronize()
    want, dot, bound = expected(g, y, w, row, kind, bs * k)
    assert np.array_equal(out.float().cpu().numpy(), want)
    assert (np.abs(gw.cpu().numpy() - dot) <= bound).all()
    assert (gw.cpu().numpy()[row < 0] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("grad", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inplace", [False, True], ids=["", "inplace"])
def test_combine_backward_many_rows(kind, grad, inplace):
    """More bytes of rows than the caches keep (their stores are another instance), against torch on the device."""
    bs, h, k, epr, ranks = 460, 16384, 7, 4, 4  # 105 MB of rows
    rng = np.random.default_rng(17)
    idx, slot, put, base, row = routes(rng, bs, k, epr, ranks, bad=0.02)
    gen = torch.Generator(device="cuda").manual_seed(17)
    g = torch.randn((bs, h), device="cuda", generator=gen).to(TYPES[grad])
    y = torch.randn((bs * k, h), device="cuda", generator=gen).to(TYPES[kind])
    w = torch.rand((bs, k), device="cuda", generator=gen)
    recv = y.clone()
    out = recv if inplace else torch.full_like(y, FILL)
    gw = torch.full((bs, k), float("nan"), device="cuda")
    log(f"combine_backward many rows {kind} grad {grad} inplace={inplace}")
    M.moe_combine_backward(g, recv, M.dtype_code(TYPES[kind]), i32(idx), w, i32(slot), i32(put), i32(base), epr, ranks,
                           out, gw)
    torch.cuda.synchronize()
    want = y.clone() if inplace else torch.full_like(y, FILL)
    for j in range(k):
        ok = torch.from_numpy(row[:, j] >= 0).cuda()
        at = torch.from_numpy(row[:, j]).cuda()[ok]
        want[at] = (w[ok, j, None] * g[ok].float()).to(TYPES[kind])
        prod = y[at].double() * g[ok].double()
        assert ((gw[ok, j] - prod.sum(1)).abs() <= (8 * -(-h // 512) + 16) * R.U * prod.abs().sum(1)).all()
        assert (gw[~ok, j] == 0).all()
    assert torch.equal(out, want)


def test_combine_backward_skips_rows_outside_the_buffers():
    """Slots that point past the buffer are skipped, and infinities or NaN in other tokens' rows stay there."""
    rng = np.random.default_rng(5)
    idx, slot, put, base, row = routes(rng, 6, 3, 4, 2, bad=0.0)
    g, y = R.to_type(rng.standard_normal((6, 72)), "bf16"), R.to_type(rng.standard_normal((18, 72)), "bf16")
    slot[2, 1], row[2, 1] = 1 << 28, -1
    slot[4, 0], row[4, 0] = -5, -1
    y[row[0]] = np.inf
    g[1, 3] = np.nan
    w = rng.random((6, 3)).astype(np.float32)
    out = torch.full((18, 72), FILL, dtype=torch.bfloat16, device="cuda")
    gw = torch.zeros((6, 3), device="cuda")
    log("combine_backward rows outside")
    M.moe_combine_backward(dev(g, "bf16"), dev(y, "bf16"), M.MOE_BF16, i32(idx), dev(w, "fp32"), i32(slot), i32(put),
                           i32(base), 4, 2, out, gw)
    torch.cuda.synchronize()
    want, dot, bound = expected(g, y, w, row, "bf16", 18)
    assert np.array_equal(out.float().cpu().numpy(), want, equal_nan=True)
    got = gw.cpu().numpy()
    assert (got[[2, 4], [1, 0]] == 0).all() and np.isnan(got[1]).all() and not np.isfinite(got[0]).any()
    rest = np.ones((6, 3), bool)
    rest[[0, 1]] = False
    assert (np.abs(got - dot)[rest] <= bound[rest]).all()


def test_combine_backward_of_several_sources():
    """Two sources' calls fill the shared buffer as two separate gradients."""
    rng = np.random.default_rng(6)
    epr, ranks, h, k, sizes = 3, 2, 136, 4, (5, 9)
    e = epr * ranks
    idxs = [rng.integers(0, e, (b, k)).astype(np.int32) for b in sizes]
    counts = np.stack([np.bincount(i.reshape(-1), minlength=e) for i in idxs])
    flat_start = (np.cumsum(counts.T.reshape(-1)) - counts.T.reshape(-1)).reshape(e, 2)  # expert-major, source-minor
    base = flat_start[::epr, 0]
    put = flat_start - np.repeat(base, epr)[:, None]
    total = sum(sizes) * k
    y = R.to_type(rng.standard_normal((total, h)), "fp16")
    out = torch.full((total, h), FILL, dtype=torch.float16, device="cuda")
    want_all = np.full((total, h), FILL, np.float32)
    for s, b in enumerate(sizes):
        slot = np.zeros((b, k), np.int32)
        seen = np.zeros(e, int)
        for i, ex in enumerate(idxs[s].reshape(-1)):
            slot.reshape(-1)[i] = seen[ex]
            seen[ex] += 1
        row = flat_start[idxs[s], s] + slot
        g, w = R.to_type(rng.standard_normal((b, h)), "fp32"), rng.random((b, k)).astype(np.float32)
        gw = torch.zeros((b, k), device="cuda")
        log(f"combine_backward source {s}")
        M.moe_combine_backward_src(dev(g, "fp32"), dev(y, "fp16"), M.MOE_FP16, i32(idxs[s]), dev(w, "fp32"), i32(slot),
                                   i32(put), i32(base), epr, ranks, s, out, gw)
        torch.cuda.synchronize()
        want, dot, bound = expected(g, y, w, row, "fp16", total)
        want_all[row.reshape(-1)] = want[row.reshape(-1)]
        assert (np.abs(gw.cpu().numpy() - dot) <= bound).all()
    assert np.array_equal(out.float().cpu().numpy(), want_all)


def test_combine_backward_matches_differences_of_combine():
    """The combine is linear in its weights and in its rows: a step of 1 in one
    weight, or of 1 in one element of a row, changes <g, out> by its gradient."""
    rng = np.random.default_rng(7)
    bs, h, k, epr, ranks = 6, 80, 3, 4, 2
    idx, slot, put, base, row = routes(rng, bs, k, epr, ranks, bad=0.0)
    y = R.to_type(np.round(rng.standard_normal((bs * k, h)) * 4), "bf16")
    g = R.to_type(np.round(rng.standard_normal((bs, h)) * 4), "fp32")
    w = (rng.integers(1, 8, (bs, k)) / 8).astype(np.float32)  # small whole numbers and eighths: every sum is exact
    ids = [i32(a) for a in (idx, slot, put, base)]

    def loss(yy, ww):
        out = torch.zeros((bs, h), device="cuda")
        M.moe_combine(dev(yy, "bf16"), M.MOE_BF16, h, ids[0], dev(ww, "fp32"), ids[1], ids[2], ids[3], epr, ranks, out)
        return float((out.double() * dev(g, "fp32").double()).sum())

    gr = torch.zeros((bs * k, h), dtype=torch.bfloat16, device="cuda")
    gw = torch.zeros((bs, k), device="cuda")
    log("combine_backward differences")
    M.moe_combine_backward(dev(g, "fp32"), dev(y, "bf16"), M.MOE_BF16, ids[0], dev(w, "fp32"), ids[1], ids[2], ids[3],
                           epr, ranks, gr, gw)
    torch.cuda.synchronize()
    at = loss(y, w)
    for t, j in ((0, 0), (3, 2), (5, 1)):
        ww = w.copy()
        ww[t, j] += 1
        assert loss(y, ww) - at == float(gw[t, j])
        for c in (0, 41, 79):
            yy = y.copy()
            yy[row[t, j], c] += 1
            assert loss(yy, w) - at == float(gr[row[t, j], c])
