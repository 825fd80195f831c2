"""The router and its gradient against their 64-bit definitions: the choice
exactly, weights and gradients within the roundings they take."""

import numpy as np
import pytest
import torch

import combine_moe_layout_03_amd as M
import router_ref as R
from gpu_util import log

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def dev(x, kind="fp32"):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(TYPES[kind])


def run_route(x, kind, k, sigmoid, bias=None, mask=None, stride=None, **kw):
    bs, e = x.shape
    if stride:
        buf = torch.full((bs, stride), float("nan"), dtype=TYPES[kind], device="cuda")
        buf[:, :e] = dev(x, kind)
        t = buf[:, :e]
    else:
        t = dev(x, kind)
    idx = torch.full((bs, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((bs, k), float("nan"), device="cuda")
    names = dict(groups="num_groups", keep="topk_groups", renorm="renormalize")
    M.moe_route(t, idx, w, M.MOE_SCORE_SIGMOID if sigmoid else M.MOE_SCORE_SOFTMAX,
                bias=None if bias is None else dev(bias),
                token_mask=None if mask is None else torch.from_numpy(mask.astype(np.uint8)).cuda(),
                **{names.get(n, n): v for n, v in kw.items()})
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def check_route(x, kind, k, sigmoid, bias=None, mask=None, stride=None, **kw):
    idx, w = run_route(x, kind, k, sigmoid, bias, mask, stride, **kw)
    want, ww, tol = R.route(x.astype(np.float64), k, sigmoid, None if bias is None else bias.astype(np.float64),
                            mask=mask, **kw)
    assert np.array_equal(idx, want), np.argwhere(idx != want)[:5]
    assert (np.abs(w - ww) <= tol * np.abs(ww) + R.TINY["fp32"] * abs(kw.get("scale", 1.0))).all(), \
        np.max(np.abs(w - ww) / np.maximum(np.abs(ww), 1e-300) / np.maximum(tol, 1e-30))
    return idx


# bs, E, k, groups, keep, group_top, bias
SHAPES = [
    (1, 256, 8, 8, 4, 2, True), (1, 1, 1, 1, 1, 1, False), (5, 2, 2, 1, 1, 1, True), (33, 64, 6, 1, 1, 1, False),
    (17, 60, 4, 1, 1, 1, True), (9, 160, 6, 8, 3, 1, False), (21, 160, 6, 8, 3, 2, True), (7, 65, 5, 5, 2, 2, False),
    (13, 128, 32, 4, 4, 1, True), (6, 512, 8, 8, 4, 2, True), (3, 513, 7, 27, 9, 1, True), (2, 1000, 10, 1, 1, 1, True),
    (2, 2048, 32, 64, 8, 2, True), (3, 2048, 16, 1, 1, 1, False), (4, 64, 8, 64, 8, 1, True), (4, 96, 8, 48, 8, 2, True),
    (257, 16, 2, 1, 1, 1, False), (5, 320, 9, 2, 1, 2, False), (130, 8, 2, 4, 1, 2, True),
    (2, 2040, 9, 24, 5, 2, True), (3, 900, 5, 12, 4, 1, True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_route_shapes(shape, sigmoid):
    bs, e, k, groups, keep, top, biased = shape
    rng = np.random.default_rng(bs * 7919 + e * 31 + k)
    for kind in ("bf16", "fp16", "fp32"):
        for renorm in (True, False):
            log(f"route {shape} {kind} sigmoid={sigmoid} renorm={renorm}")
            check_route(R.logits(rng, bs, e, kind), kind, k, sigmoid,
                        (rng.standard_normal(e) * 0.05).astype(np.float32) if biased else None, groups=groups,
                        keep=keep, group_top=top, renorm=renorm, scale=2.5)


# Batches that take four tokens a wave: E, k, groups, keep, group_top, bias
LARGE = [(8, 2, 1, 1, 1, False), (16, 8, 4, 2, 1, True), (16, 16, 1, 1, 1, True), (30, 3, 5, 2, 2, False), (64, 6, 8, 3, 2, True),
         (100, 7, 4, 2, 2, True), (128, 8, 1, 1, 1, True), (160, 6, 8, 3, 1, False), (256, 8, 8, 4, 2, True),
         (256, 16, 64, 9, 2, True), (256, 1, 2, 1, 2, False)]


@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
def test_route_large_batches(shape, sigmoid):
    e, k, groups, keep, top, biased = shape
    rng = np.random.default_rng(e + k)
    kind = ("bf16", "fp16", "fp32")[(e + k) % 3]
    x = R.logits(rng, 4101, e, kind)
    x[5], x[6, : e // 2], x[4100] = -np.inf, np.nan, 0.0
    mask = (rng.random(4101) > 0.1).astype(np.uint8)
    bias = (rng.standard_normal(e) * 0.05).astype(np.float32) if biased else None
    for renorm in (True, False):
        log(f"route large {shape} {kind} sigmoid={sigmoid} renorm={renorm}")
        check_route(x, kind, k, sigmoid, bias, mask, stride=e + 3, groups=groups, keep=keep, group_top=top,
                    renorm=renorm, scale=1.5)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_go_to_the_lower_id(sigmoid, biased):
    rng = np.random.default_rng(11)
    x = np.round(rng.standard_normal((64, 96))).astype(np.float32)
    x[0] = 0.0
    x[1, ::2] = -0.0  # zeros of both signs are equal
    x[1, 1::2] = 0.0
    bias = np.zeros(96, np.float32) if biased else None
    for groups, keep, top in ((1, 1, 1), (8, 2, 1), (8, 3, 2)):
        log(f"route ties sigmoid={sigmoid} bias={biased} groups={groups}")
        idx = check_route(x, "fp32", 12, sigmoid, bias, groups=groups, keep=keep, group_top=top)
        assert idx[0, 0] == 0 and list(idx[1, :3]) == [0, 1, 2]


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masks_and_extremes(sigmoid, renorm):
    rng = np.random.default_rng(12)
    x = R.logits(rng, 24, 72, "fp32")
    low = np.finfo(np.float32).min
    x[0] = np.nan
    x[1] = -np.inf
    x[2, 3:] = -np.inf                    # fewer eligible than k
    x[3] = low                            # a mask of the type's lowest value everywhere
    x[4, 5:] = low
    x[5, 7] = np.inf
    x[6, [9, 40]] = np.inf
    x[7] -= 200.0                         # scores that underflow
    x[8] += 200.0
    x[9, ::3] = np.nan
    x[10] = 0.0
    x[11] = -np.float32(1e-40)
    x[12, :] = -1000.0
    x[12, 70] = 1000.0
    mask = np.ones(24, np.uint8)
    mask[13:16] = 0
    x[13], x[14] = np.nan, np.inf
    bias = (rng.standard_normal(72) * 0.1).astype(np.float32)
    for b in (None, bias):
        for groups, keep, top in ((1, 1, 1), (9, 4, 1), (9, 4, 2)):
            log(f"route extremes sigmoid={sigmoid} renorm={renorm} bias={b is not None} groups={groups}")
            idx = check_route(x, "fp32", 8, sigmoid, b, mask, groups=groups, keep=keep, group_top=top, renorm=renorm)
            assert (idx[[0, 1, 13, 14, 15]] == -1).all() and (idx[2, 3:] == -1).all()


def test_route_large_bias_is_clipped():
    x = R.logits(np.random.default_rng(13), 4, 30, "fp32")
    bias = np.zeros(30, np.float32)
    bias[[3, 9]] = 1e9
    bias[[5, 6]] = -1e9
    log("route clipped bias")
    idx = check_route(x, "fp32", 30, True, bias)
    assert (idx[:, :2] == [3, 9]).all() and (idx[:, -2:] == [5, 6]).all()


@pytest.mark.parametrize("kind,stride", [("fp32", 61), ("bf16", 61), ("fp16", 97), ("fp32", 64)])
def test_route_row_strides(kind, stride):
    x = R.logits(np.random.default_rng(14), 19, 60, kind)
    log(f"route stride {stride} {kind}")
    check_route(x, kind, 5, True, np.zeros(60, np.float32), stride=stride, groups=4, keep=2, group_top=2)


def test_route_offset_rows_and_empty_batch():
    """Logits that start at an odd element, and a batch of no tokens."""
    x = R.logits(np.random.default_rng(15), 9, 33, "bf16")
    buf = torch.zeros(9 * 33 + 1, dtype=torch.bfloat16, device="cuda")
    buf[1:] = dev(x, "bf16").view(-1)
    idx = torch.zeros((9, 4), dtype=torch.int32, device="cuda")
    w = torch.zeros((9, 4), device="cuda")
    log("route odd offset")
    M.moe_route(buf[1:].view(9, 33), idx, w, M.MOE_SCORE_SOFTMAX)
    torch.cuda.synchronize()
    assert np.array_equal(idx.cpu().numpy(), R.route(x.astype(np.float64), 4, False)[0])
    M.moe_route(torch.zeros((0, 33), device="cuda"), idx[:0], w[:0], M.MOE_SCORE_SOFTMAX)


def check_backward(x, kind, idx, sigmoid, renorm, scale=2.5, seed=0, stride=None):
    bs, e = x.shape
    g = np.random.default_rng(seed + 99).standard_normal(idx.shape).astype(np.float32)
    t = dev(x, kind)
    width = stride or e
    buf = torch.full((bs, width), float("nan"), dtype=TYPES[kind], device="cuda")
    M.moe_route_backward(dev(g), t, torch.from_numpy(np.ascontiguousarray(idx, np.int32)).cuda(),
                         M.MOE_SCORE_SIGMOID if sigmoid else M.MOE_SCORE_SOFTMAX, buf[:, :e], renormalize=renorm,
                         scale=scale)
    torch.cuda.synchronize()
    got = buf[:, :e].float().cpu().numpy().astype(np.float64)
    assert stride is None or torch.isnan(buf[:, e:]).all()
    want, mag = R.route_backward(g, x.astype(np.float64), idx, sigmoid, renorm, scale)
    # a share or a score is off by at most (2 (4 + d) + 40) U (see router_ref.route), d <= 200; it enters a
    # term at most three times, and the sums, products and the slope add at most 60 roundings
    ok = R.eligible(x.astype(np.float64))
    y = np.where(ok, np.clip(x, -200, 200), 0).astype(np.float64)
    d = np.minimum(y.max(axis=1) - np.where(ok, y, np.inf).min(axis=1, initial=np.inf), 200.0)
    d = np.where(np.isfinite(d), np.maximum(d, np.abs(y).max(axis=1)), 0.0)[:, None]
    tol = (3 * (2 * (4 + d) + 40) + 60) * R.U * mag
    bound = tol + R.HALF_STEP[kind] * (np.abs(want) + tol) + R.TINY[kind]
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / bound)


@pytest.mark.parametrize("bs,e,k", [(1, 256, 8), (5, 1, 1), (33, 64, 6), (9, 160, 6), (6, 513, 32), (2, 2048, 16),
                                    (130, 8, 2), (3, 60, 30)])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(bs, e, k, sigmoid, renorm):
    rng = np.random.default_rng(bs + e + k)
    for kind in ("bf16", "fp16", "fp32"):
        x = R.logits(rng, bs, e, kind)
        idx = np.stack([rng.permutation(e)[:k] for _ in range(bs)]).astype(np.int32)
        log(f"route_backward {bs} {e} {k} {kind} sigmoid={sigmoid} renorm={renorm}")
        check_backward(x, kind, idx, sigmoid, renorm, seed=k)


@pytest.mark.parametrize("e,k", [(8, 2), (17, 16), (60, 5), (100, 7), (128, 8), (256, 8)])
@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_large_batches(e, k, sigmoid, renorm):
    rng = np.random.default_rng(e * k)
    kind = ("bf16", "fp16", "fp32")[(e + k) % 3]
    x = R.logits(rng, 4101, e, kind)
    idx = np.argsort(rng.random((4101, e)), axis=1)[:, :k].astype(np.int32)
    x[7], idx[7], idx[4100, 1:] = np.nan, -1, -1
    log(f"route_backward large {e} {k} {kind} sigmoid={sigmoid} renorm={renorm}")
    check_backward(x, kind, idx, sigmoid, renorm, stride=e + 5)


@pytest.mark.parametrize("sigmoid", [False, True], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_extremes(sigmoid, renorm):
    """Masked tokens (ids -1, anything in the logits), experts that are not
    eligible, ids outside the range, underflowing scores, a strided output."""
    rng = np.random.default_rng(21)
    x = R.logits(rng, 12, 50, "fp32")
    idx = np.stack([rng.permutation(50)[:6] for _ in range(12)]).astype(np.int32)
    x[0], idx[0] = np.nan, -1
    x[1], idx[1] = np.inf, -1
    idx[2, 3:] = -1
    idx[3, 0], idx[3, 1] = 50, -2147483648
    x[4, ::4] = -np.inf
    x[5, idx[5, 2]] = np.nan
    x[6] -= 150.0
    x[7] += 150.0
    x[8] = np.finfo(np.float32).min
    x[9] = -np.inf
    log(f"route_backward extremes sigmoid={sigmoid} renorm={renorm}")
    check_backward(x, "fp32", idx, sigmoid, renorm, stride=53)


def test_route_on_another_stream_and_in_a_graph():
    """Both calls on a side stream, then captured and replayed on new logits
    with eager calls between, every replay against the eager result."""
    rng = np.random.default_rng(31)
    xs = [dev(R.logits(rng, 40, 64, "fp32")) for _ in range(3)]
    x = xs[0].clone()
    idx = torch.zeros((40, 4), dtype=torch.int32, device="cuda")
    w, g = torch.zeros((40, 4), device="cuda"), torch.randn((40, 4), device="cuda")
    dx = torch.zeros_like(x)

    def step(stream=None):
        M.moe_route(x, idx, w, M.MOE_SCORE_SIGMOID, num_groups=4, topk_groups=2, group_top=2, stream=stream)
        M.moe_route_backward(g, x, idx, M.MOE_SCORE_SIGMOID, dx, stream=stream)

    want = []
    for q in xs:
        x.copy_(q)
        step()
        torch.cuda.synchronize()
        want.append((idx.clone(), w.clone(), dx.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    log("route side stream")
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((idx, w, dx), want[2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r, q in enumerate(xs * 2):
        x.copy_(q)
        for o in (idx, w, dx):
            o.zero_()
        torch.cuda.synchronize()
        log(f"route graph replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((idx, w, dx), want[r % 3]))
        M.moe_route(x, idx, w, M.MOE_SCORE_SOFTMAX)
        torch.cuda.synchronize()
