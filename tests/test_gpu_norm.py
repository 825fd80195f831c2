"""The root-mean-square norm, its 8-bit rows and its gradient against 64 bits."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log

pytestmark = pytest.mark.gpu


def host(t):
    return t.detach().float().cpu().double().numpy()


def make(rng, bs, h, kind, spread=3.0):
    v = rng.normal(size=(bs, h)) * np.exp(rng.normal(size=(bs, 1)) * spread / 3)
    return torch.from_numpy(v).to(B.TYPES[kind]).cuda()


def run(x, res, w, eps, out_kind, rows, rstd, in_place=False):
    bs, h = x.shape
    s = None if res is None else (res if in_place else torch.full_like(x, 7))
    out = None if out_kind is None else torch.full((bs, h), 7, dtype=B.TYPES[out_kind], device="cuda")
    buf = torch.full((bs * B.row_bytes(h),), 0xA5, dtype=torch.uint8, device="cuda") if rows else None
    r = torch.zeros(bs, device="cuda") if rstd else None
    M.moe_rms_norm(x, w, eps, residual=res, sum=s, out=out, rows=buf, rstd=r)
    torch.cuda.synchronize()
    return s, out, buf, r


def check(rng, bs, h, kind, out_kind="bf16", res=True, rows=True, rstd=True, eps=1e-6, in_place=False):
    log(f"rms_norm {bs} {h} {kind} -> {out_kind} residual {res} rows {rows} in place {in_place}")
    x = make(rng, bs, h, kind)
    r = make(rng, bs, h, kind) if res else None
    w = torch.from_numpy((rng.random(h) + 0.5).astype(np.float32)).cuda()
    kept = (x.float() + r.float()).to(x.dtype) if res else x.clone()
    s, out, buf, rs = run(x, r, w, eps, out_kind, rows, rstd, in_place)
    if res:
        assert torch.equal(s, kept)
    y, want_rstd = B.norm(host(kept), host(w), eps)
    if out is not None:
        assert B.near(host(out), y, out_kind, B.NORM * np.abs(y))
    if rstd:
        assert (np.abs(host(rs) - want_rstd) <= B.RSTD * want_rstd).all()
    if rows:
        B.check_rows(*B.unpack(buf, bs, h), y, B.NORM * np.abs(y))
        assert (B.padding(buf, bs, h) == 0xA5).all()


@pytest.mark.parametrize("h", [16, 32, 112, 128, 144, 512, 528, 1024, 1040, 2064, 4096, 7168, 8192, 8208, 16384])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_norm_widths(h, kind):
    rng = np.random.default_rng(h)
    for bs in (1, 5):
        check(rng, bs, h, kind, out_kind={"bf16": "bf16", "fp16": "fp32", "fp32": "fp16"}[kind])


@pytest.mark.parametrize("bs", [1, 2, 3, 4, 7, 64, 257, 1025])
@pytest.mark.parametrize("h", [8, 24, 504, 1000, 2040])
def test_norm_batches_without_rows(bs, h):
    check(np.random.default_rng(bs + h), bs, h, "bf16", out_kind="bf16", rows=False)


@pytest.mark.parametrize("out_kind", ["bf16", "fp16", "fp32", None])
@pytest.mark.parametrize("res", [True, False])
def test_norm_outputs(out_kind, res):
    rng = np.random.default_rng(3)
    for kind in ("bf16", "fp16", "fp32"):
        for h in (304, 2064):
            check(rng, 9, h, kind, out_kind=out_kind, res=res, rstd=res)


def test_norm_in_place_sum():
    rng = np.random.default_rng(4)
    for kind in ("bf16", "fp16", "fp32"):
        check(rng, 33, 1040, kind, in_place=True)
    x, r = make(rng, 6, 256, "bf16"), make(rng, 6, 256, "bf16")
    want = (x.float() + r.float()).bfloat16()
    out = torch.zeros_like(x)
    M.moe_rms_norm(x, torch.ones(256, device="cuda"), 1e-6, residual=r, sum=x, out=out)  # over x instead
    torch.cuda.synchronize()
    assert torch.equal(x, want)


def test_norm_zeros_tiny_and_extreme_rows():
    """Rows of zeros (codes 0 and the least scale), rows whose squares are subnormal, and rows near the largest value."""
    rng = np.random.default_rng(5)
    h = 400
    x = torch.from_numpy(rng.normal(size=(5, h))).float().cuda()
    x[0] = 0
    x[1] *= 1e-15
    x[2, :128] = 0
    x[3] *= 1e17
    w = torch.ones(h, device="cuda")
    for eps in (1e-6, 1e-30):
        log(f"rms_norm extremes eps {eps}")
        _, out, buf, rs = run(x, None, w, eps, "fp32", True, True)
        y, _ = B.norm(host(x), np.ones(h), eps)
        assert B.near(host(out), y, "fp32", B.NORM * np.abs(y))
        codes, scales = B.unpack(buf, 5, h)
        B.check_rows(codes, scales, y, B.NORM * np.abs(y))
        assert (codes[0] == 0).all() and (np.abs(scales[0] * 448 / 2.0 ** -100 - 1) <= 2 * B.U).all()
        assert (codes[2, :128] == 0).all() and (out[0] == 0).all()


def test_norm_not_finite_rows_stay_alone():
    rng = np.random.default_rng(6)
    x = make(rng, 6, 272, "bf16")
    x[1, 5], x[4, 200] = float("nan"), float("inf")
    w = torch.ones(272, device="cuda")
    log("rms_norm rows that are not finite")
    _, out, buf, _ = run(x, None, w, 1e-6, "bf16", True, False)
    keep = [0, 2, 3, 5]
    y, _ = B.norm(host(x)[keep], np.ones(272), 1e-6)
    assert B.near(host(out)[keep], y, "bf16", B.NORM * np.abs(y))
    codes, scales = B.unpack(buf, 6, 272)
    B.check_rows(codes[keep], scales[keep], y, B.NORM * np.abs(y))
    assert torch.isnan(out[1]).all() and np.isnan(codes[1]).all()
    bad = torch.isnan(out[4]).cpu().numpy()
    assert bad[200] and bad.sum() == 1 and (out[4][~torch.isnan(out[4])] == 0).all() and np.isnan(codes[4, 200])


def test_norm_empty_batch_and_streams():
    w = torch.ones(64, device="cuda")
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    M.moe_rms_norm(x, w, 1e-6, out=torch.zeros_like(x))
    rng = np.random.default_rng(7)
    x, out = make(rng, 40, 64, "bf16"), torch.zeros((40, 64), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    log("rms_norm on another stream")
    M.moe_rms_norm(x, w, 1e-6, out=out, stream=side)
    side.synchronize()
    y, _ = B.norm(host(x), np.ones(64), 1e-6)
    assert B.near(host(out), y, "bf16", B.NORM * np.abs(y))


def test_norm_e4m3_conversion_of_every_value():
    """Every e4m3 magnitude, the middles between neighbours and the floats beside them, through a block whose factor
    is 1: the largest is 448."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    every = np.sort(every[np.isfinite(every)])
    mid = ((every[1:].astype(np.float64) + every[:-1]) / 2).astype(np.float32)
    v = np.concatenate([every, mid, np.nextafter(mid, np.float32(500)), np.nextafter(mid, np.float32(-500))])
    v = np.resize(v, (v.size + 126) // 127 * 127).reshape(-1, 127)
    v = np.concatenate([v, np.full((v.shape[0], 1), 448, np.float32)], axis=1)
    # one row of 128 values and so many of 0 that the mean of squares plus eps can be made 1: rstd is then exact
    x = torch.from_numpy(v).cuda()
    mean = (v.astype(np.float64) ** 2).mean(axis=1)
    # w undoes rstd up to its error; the largest stays 448 in y up to it too, so the factor undoes the rest
    log("rms_norm e4m3 conversion")
    for r in range(x.shape[0]):
        w = torch.full((128,), float(np.sqrt(mean[r])), device="cuda")
        _, _, buf, _ = run(x[r:r + 1].contiguous(), None, w, 0.0, None, True, False)
        codes, scales = B.unpack(buf, 1, 128)
        y = host(x[r:r + 1])
        B.check_rows(codes, scales, y, (B.NORM + 2 * B.U) * np.abs(y))


# ---- gradient ----------------------------------------------------------------------


def check_backward(rng, bs, h, kind, grad="bf16", skip=True, weight=True, mask=None, in_place=None):
    log(f"rms_norm_backward {bs} {h} {kind} {grad} skip {skip} weight {weight} in place {in_place}")
    s = make(rng, bs, h, kind)
    g = make(rng, bs, h, grad, 1.0)
    k = make(rng, bs, h, kind, 1.0) if skip else None
    w = torch.from_numpy((rng.random(h) + 0.5).astype(np.float32)).cuda()
    _, rstd = B.norm(host(s), host(w), 1e-6)
    rstd = torch.from_numpy(rstd).float().cuda()
    gh, sh, kh = host(g), host(s), host(k) if skip else None
    tm = None
    if mask is not None:
        gh, sh = np.where(mask[:, None], gh, 0), np.where(mask[:, None], sh, 0)
        kh = np.where(mask[:, None], kh, 0) if skip else None
        s[torch.from_numpy(~mask).cuda()] = float("nan")
        rstd[torch.from_numpy(~mask).cuda()] = float("nan")
        tm = torch.from_numpy(mask.astype(np.uint8)).cuda()
    dx = {"skip": k, "grad": g}.get(in_place)
    dx = torch.full_like(s, 7) if dx is None else dx
    dw = torch.full((h,), 7.0, device="cuda") if weight else None
    ws = torch.full((M.moe_rms_norm_backward_workspace_bytes(bs, h),), 0xFF, dtype=torch.uint8, device="cuda")
    M.moe_rms_norm_backward(g, s, w, rstd, dx, grad_sum=k, grad_weight=dw, workspace=ws if weight else None,
                            token_mask=tm)
    torch.cuda.synchronize()
    want, err, want_w, err_w = B.norm_backward(gh, sh, host(w), np.nan_to_num(host(rstd)), kh)
    assert B.near(host(dx), want, kind, err)
    if mask is not None:
        assert (host(dx)[~mask] == 0).all()
    if weight:
        assert (np.abs(host(dw) - want_w) <= err_w + 2.0 ** -140).all()


@pytest.mark.parametrize("h", [8, 24, 504, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 7168, 8192, 8200, 16384])
def test_norm_backward_widths(h):
    rng = np.random.default_rng(h)
    for bs in (1, 6):
        check_backward(rng, bs, h, "bf16")


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("grad", ["bf16", "fp16", "fp32"])
def test_norm_backward_types(kind, grad):
    rng = np.random.default_rng(8)
    for h in (256, 1000, 2064, 16376):
        check_backward(rng, 11, h, kind, grad, skip=h != 256)


@pytest.mark.parametrize("bs", [1, 3, 4, 255, 511, 512, 513, 1030, 2100])
def test_norm_backward_batches(bs):
    rng = np.random.default_rng(bs)
    for h in (72, 1032):
        check_backward(rng, bs, h, "fp32", "fp32", skip=False)


def test_norm_backward_masks_in_place_and_frozen_weight():
    rng = np.random.default_rng(9)
    for h in (136, 1160):
        check_backward(rng, 37, h, "bf16", mask=rng.random(37) < 0.6)
        check_backward(rng, 8, h, "bf16", mask=np.zeros(8, bool))
        check_backward(rng, 37, h, "bf16", in_place="skip")
        check_backward(rng, 37, h, "fp16", "fp16", in_place="grad")
        check_backward(rng, 37, h, "fp32", weight=False)


def test_norm_backward_empty_batch_writes_zeros():
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), 7.0, device="cuda")
    e = torch.zeros((0, 64), device="cuda")
    log("rms_norm_backward of an empty batch")
    M.moe_rms_norm_backward(e, e, w, torch.zeros(0, device="cuda"), torch.zeros_like(e), grad_weight=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_norm_backward_same_result_twice_and_on_replays():
    """The weight's gradient does not depend on scheduling, and a captured step replays on new inputs."""
    rng = np.random.default_rng(10)
    bs, h = 700, 520
    s, g, w = make(rng, bs, h, "bf16"), make(rng, bs, h, "bf16"), torch.ones(h, device="cuda")
    rstd, out = torch.zeros(bs, device="cuda"), torch.zeros_like(s)
    dx, dw = torch.zeros_like(s), torch.zeros(h, device="cuda")
    ws = torch.zeros(M.moe_rms_norm_backward_workspace_bytes(bs, h), dtype=torch.uint8, device="cuda")

    def step():
        M.moe_rms_norm(s, w, 1e-6, out=out, rstd=rstd)
        M.moe_rms_norm_backward(g, s, w, rstd, dx, grad_weight=dw, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        s.copy_(make(rng, bs, h, "bf16"))
        log(f"rms_norm replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in (out, rstd, dx, dw)]
        for t in (out, rstd, dx, dw):
            t.fill_(3)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (out, rstd, dx, dw)))


def test_norm_backward_against_differences():
    """The gradient of a scalar of the forward's own outputs along random directions."""
    rng = np.random.default_rng(11)
    bs, h = 6, 264
    s, g, w = rng.normal(size=(bs, h)), rng.normal(size=(bs, h)), rng.random(h) + 0.5
    ts, tg, tw = (torch.from_numpy(v).float().cuda() for v in (s, g, w))
    s, g, w = host(ts), host(tg), host(tw)
    rstd, out = torch.zeros(bs, device="cuda"), torch.zeros_like(ts)
    M.moe_rms_norm(ts, tw, 1e-5, out=out, rstd=rstd)
    dx, dw = torch.zeros_like(ts), torch.zeros(h, device="cuda")
    ws = torch.zeros(M.moe_rms_norm_backward_workspace_bytes(bs, h), dtype=torch.uint8, device="cuda")
    M.moe_rms_norm_backward(tg, ts, tw, rstd, dx, grad_weight=dw, workspace=ws)
    torch.cuda.synchronize()
    for _ in range(3):
        d, e, step = rng.normal(size=s.shape), rng.normal(size=h), 1e-5
        slope = ((B.norm(s + step * d, w + step * e, 1e-5)[0] - B.norm(s - step * d, w - step * e, 1e-5)[0]) * g).sum()
        got = (host(dx) * d).sum() + (host(dw) * e).sum()
        # the differences are off by about step^2, the gradients by some 70 roundings of their terms
        bound = 70 * B.U * ((np.abs(g) * w).sum() * 4 + np.abs(host(dw) * e).sum() + np.abs(host(dx) * d).sum()) + 1e-6
        assert abs(slope / (2 * step) - got) <= bound


@pytest.mark.parametrize("kind,bs,h", [("bf16", 4100, 7168), ("fp32", 1700, 8208), ("fp16", 900, 16384), ("fp32", 30000, 1040)])
def test_norm_large_batches(kind, bs, h):
    """Batches of more than the caches keep (their rows are loaded in another way), some rows of each."""
    log(f"rms_norm large {kind} {bs} {h}")
    gen = torch.Generator(device="cuda").manual_seed(h)
    x, r, g, k = (torch.randn((bs, h), device="cuda", generator=gen).to(B.TYPES[kind]) for _ in range(4))
    w = torch.rand(h, device="cuda", generator=gen) + 0.5
    s, out, buf, rstd = run(x, r, w, 1e-6, kind, True, True)
    assert torch.equal(s, (x.float() + r.float()).to(x.dtype))
    some = sorted({0, 1, bs // 2, bs - 2, bs - 1} | set(np.random.default_rng(h).integers(0, bs, 20).tolist()))
    y, want = B.norm(host(s[some]), host(w), 1e-6)
    assert B.near(host(out[some]), y, kind, B.NORM * np.abs(y)) and (np.abs(host(rstd[some]) - want) <= B.RSTD * want).all()
    B.check_rows(*B.unpack(buf.view(bs, -1)[some].contiguous(), len(some), h), y, B.NORM * np.abs(y))
    dx, dw = torch.full_like(s, 7), torch.full((h,), 7.0, device="cuda")
    ws = torch.full((M.moe_rms_norm_backward_workspace_bytes(bs, h),), 0xFF, dtype=torch.uint8, device="cuda")
    M.moe_rms_norm_backward(g, s, w, rstd, dx, grad_sum=k, grad_weight=dw, workspace=ws)
    torch.cuda.synchronize()
    dxs, err, _, _ = B.norm_backward(host(g[some]), host(s[some]), host(w), host(rstd[some]), host(k[some]))
    assert B.near(host(dx[some]), dxs, kind, err)
    terms = g.double() * s.double() * rstd.double()[:, None]
    bound = (bs + 8) * B.U * terms.abs().sum(dim=0)
    assert ((dw.double() - terms.sum(dim=0)).abs() <= bound).all()
