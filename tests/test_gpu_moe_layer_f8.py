"""A whole layer in 8-bit floats, each stage against 64 bits on what the stage
before it left, and the norm in front of a training layer."""

import os
import runpy

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    return runpy.run_path(os.path.join(ROOT, "examples", "moe_layer.py"))


def host(t):
    return t.detach().float().cpu().double().numpy()


def check_stages(layer, x, residual, bs):
    """Every stage of the step that `layer` has just made, from its own buffers."""
    h, n, topk, experts = layer.hidden, layer.n, layer.idx.shape[1], layer.w2.shape[0]
    # the norm
    kept = (x.float() + residual.float()).to(x.dtype)
    assert torch.equal(layer.sum[:bs], kept)
    y, _ = B.norm(host(kept), host(layer.norm_weight), 1e-6)
    assert B.near(host(layer.normed[:bs]), y, "bf16", B.NORM * np.abs(y))
    B.check_rows(*B.unpack(layer.token_rows[:bs].contiguous(), bs, h), y, B.NORM * np.abs(y))
    # the dispatch: every routed row as it is, sorted by expert
    idx = layer.idx[:bs].cpu().numpy()
    order = [(e, t) for e in range(experts) for t, j in zip(*np.nonzero(idx == e))]
    rows = len(order)
    recv = layer.ep.recv_x.view(-1, layer.ep.row_bytes)
    a, ts = B.unpack(layer.ep.recv_x, recv.shape[0], h)
    ta, tts = B.unpack(layer.token_rows, layer.token_rows.shape[0], h)
    of = [t for _, t in order]
    assert np.array_equal(a[:rows], ta[of]) and np.array_equal(ts[:rows], tts[of])
    # the first product and its gate
    own = np.array([e for e, _ in order])
    y, err = B.product(a[:rows], ts[:rows], host(layer.w1), host(layer.w1_scale), own, n)
    act, err = B.gated(y, err, n)
    q, qs = B.unpack(layer.act, layer.rows, n)
    B.check_rows(q[:rows], qs[:rows], act, err)
    # the second product
    w2, s2 = host(layer.w2), host(layer.w2_scale)
    y, err = B.product(q[:rows], qs[:rows], w2, s2, own, h)
    got = host(layer.out_rows)[:rows]
    assert B.near(got, y, "bf16", err + B.cut(q[:rows], qs[:rows], w2, s2, own, h))
    # the combine, in entry order
    place = {(e, t): r for r, (e, t) in enumerate(order)}
    weights = host(layer.weights)
    want = np.zeros((bs, h))
    size = np.zeros((bs, h))
    for t in range(bs):
        for j in range(topk):
            if idx[t, j] >= 0:
                v = weights[t, j] * got[place[idx[t, j], t]]
                want[t] += v
                size[t] += np.abs(v)
    assert B.near(host(layer.out[:bs]), want, "bf16", 2 * topk * B.U * size)


def test_float8_layer(example):
    log("8-bit float layer")
    out, ref, layer = example["float8_example"]()
    assert (out[3] == 0).all()  # the masked token has no expert
    # a rounding to e4m3 is off by 2^-4 at most, and by less than 2^-4 / sqrt(3) = 0.036 in the mean square; rows and
    # weights are rounded in two products, the first of which counts twice (gate and up): sqrt(2 * 2 + 2) of it, 0.088
    assert float((out - ref).norm() / ref.norm()) < 0.1


@pytest.mark.parametrize("tokens,hidden,n,experts,topk", [(1, 256, 128, 8, 2), (48, 256, 160, 16, 4), (700, 512, 144, 8, 2)])
def test_float8_layer_stage_by_stage(example, tokens, hidden, n, experts, topk):
    log(f"8-bit float layer stages {tokens} {hidden} {n} {experts} {topk}")
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    blocks = example["quantised_blocks"]
    w1, w2 = rand(experts, 2 * n, hidden) / hidden ** 0.5, rand(experts, hidden, n) / n ** 0.5
    (g, gs), (u, us), (q2, s2) = blocks(w1[:, :n]), blocks(w1[:, n:]), blocks(w2)
    layer = example["Float8Layer"](tokens, topk, 0.5 + torch.rand(hidden, device="cuda", generator=gen),
                                   torch.cat([g, u], dim=1), torch.cat([gs, us], dim=1), q2, s2,
                                   rand(experts, hidden) / hidden ** 0.5, rand(experts) * 0.05, 4, 2, 2.5)
    for bs in {tokens, max(1, tokens // 2)}:  # a smaller batch in the same buffers too
        x, residual = rand(bs, hidden).bfloat16(), rand(bs, hidden).bfloat16()
        layer.step(x, residual)
        torch.cuda.synchronize()
        check_stages(layer, x, residual, bs)


def test_float8_layer_replays(example):
    """A captured step on new tokens, with eager steps of another layer between the replays."""
    out, ref, layer = example["float8_example"]()
    _, _, other = example["float8_example"](seed=5)
    bs = 48
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((bs, layer.hidden), device="cuda", generator=gen).bfloat16()
    residual = torch.randn((bs, layer.hidden), device="cuda", generator=gen).bfloat16()
    layer.step(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, residual)
    for r in range(3):
        x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
        log(f"8-bit float layer replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        check_stages(layer, x, residual, bs)
        first = layer.out.clone()
        other.step(x, residual)
        layer.step(x, residual)
        torch.cuda.synchronize()
        assert torch.equal(first, layer.out)


def test_dispatch_of_e4m3_rows_several_sources():
    """e4m3 rows of two sources into one buffer, by the calls for several sources and by the stages of one."""
    hidden, topk, epr, ranks = 400, 3, 2, 4
    rng = np.random.default_rng(1)
    sizes = [7, 300]
    rb = M.moe_recv_row_bytes(hidden, M.MOE_E4M3_BLOCKSCALE)
    xs = [torch.from_numpy(rng.integers(0, 256, (b, rb), dtype=np.uint8)).cuda() for b in sizes]
    idxs = [torch.from_numpy(np.array([rng.permutation(epr * ranks)[:topk] for _ in range(b)], np.int32)).cuda()
            for b in sizes]
    buf = M.EpMultiBuffers(sizes, hidden, topk, epr, ranks, x_dtype=torch.float8_e4m3fn, quant_int8=False)
    assert buf.row_bytes == rb
    log("dispatch of e4m3 rows, two sources")
    for s in range(2):
        buf.layout(s, idxs[s])
    buf.notify()
    for s in range(2):
        buf.dispatch(s, xs[s], idxs[s])
    torch.cuda.synchronize()
    want = [xs[s][t] for e in range(epr * ranks) for s in range(2) for t in (idxs[s] == e).any(dim=1).nonzero()[:, 0]]
    assert torch.equal(buf.recv_x.view(-1, rb), torch.stack(want))
    for one_launch in (False, True):
        ep = M.EpBuffers(sizes[1], hidden, topk, epr, ranks, x_dtype=torch.float8_e4m3fn, quant_int8=False)
        log(f"dispatch of e4m3 rows, one launch {one_launch}")
        if one_launch:
            ep.layout_notify_dispatch(xs[1], idxs[1])
        else:
            ep.layout(idxs[1])
            ep.notify()
            ep.dispatch(xs[1], idxs[1])
        torch.cuda.synchronize()
        want = [xs[1][t] for e in range(epr * ranks) for t in (idxs[1] == e).any(dim=1).nonzero()[:, 0]]
        assert torch.equal(ep.recv_x.view(-1, rb), torch.stack(want))


def test_training_behind_a_norm(example):
    log("training behind a norm")
    got, ref = example["normed_training_example"]()
    for a, b in zip(got, ref):
        # sums, normed rows, expert rows, their gradients and the results are rounded to bf16, six times at most
        assert float((a.double() - b).norm() / b.norm()) < 6 * 2.0 ** -8
