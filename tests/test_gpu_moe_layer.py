"""The router, the expert products and the gradients as a layer uses them
(examples/moe_layer.py): the serving layer's pieces bit for bit and its result
near the unquantised layer, captured in a graph; the training layer's
gradients against autograd in 64 bits."""

import os
import sys

import numpy as np
import pytest
import torch

import combine_moe_layout_03_amd as M
import oracle
from gpu_util import align32, log

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def test_serving_layer():
    log("moe layer: serving")
    out, ref, layer = moe_layer.serving_example()
    torch.cuda.synchronize()
    # quantising rows, weights and activations to int8: each value is off by at most half a code of 127 in its row's
    # largest, about 1 % of the row's root mean square; three such, and the bf16 rows, stay below 5 % together
    assert float((out - ref).norm() / ref.norm()) < 0.05
    assert (out[3] == 0).all() and (layer.idx[3] == -1).all()
    # the second product's rows from the first's int8 rows, bit for bit
    raw = layer.act.cpu().numpy().reshape(layer.rows, layer.act_bytes)
    n = layer.n
    codes = np.ascontiguousarray(raw[:, :n]).view(np.int8)
    scale = np.ascontiguousarray(raw[:, align32(n):align32(n) + 4]).view(np.float32)
    acc, grp = oracle.grouped_gemm_i8(codes, n, layer.ep.recv_token_per_expert.cpu().numpy(), layer.w2.cpu().numpy())
    want = torch.from_numpy(acc.astype(np.float32) * layer.w2_scale.cpu().numpy()[np.maximum(grp, 0)] * scale).bfloat16()
    assert torch.equal(layer.out_rows.cpu()[grp >= 0], want[grp >= 0])


def test_serving_layer_in_a_graph():
    """A captured step replayed on other tokens, with eager steps of another layer between replays."""
    _, _, layer = moe_layer.serving_example(tokens=20, seed=5)
    _, _, other = moe_layer.serving_example(tokens=9, seed=6)
    gen = torch.Generator(device="cuda").manual_seed(7)
    xs = [torch.randn((20, layer.hidden), device="cuda", generator=gen).bfloat16() for _ in range(3)]
    x = xs[0].clone()
    want = [layer.step(q).clone() for q in xs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    log("moe layer: capture")
    with torch.cuda.graph(graph):
        layer.step(x)
    for r, (q, w) in enumerate(zip(xs * 2, want * 2)):
        x.copy_(q)
        layer.out.fill_(7.0)
        torch.cuda.synchronize()
        log(f"moe layer: replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, w)
        other.step(x[:9, :other.hidden].contiguous())
        torch.cuda.synchronize()


def test_training_layer_gradients():
    """Rows, row gradients and the experts' products are rounded to bf16, 2^-8 of a value each: the output and the
    gradients of x and w take at most three such roundings, the logits' gradient (a difference of weight gradients
    that took two, each a sum over h of products near its own size) a few times that."""
    log("moe layer: training")
    got, ref = moe_layer.training_example()
    torch.cuda.synchronize()
    for name, a, b, tol in zip(("out", "x", "logits", "w"), got, ref, (3, 3, 12, 3)):
        err = float((a.double() - b).norm() / b.norm())
        log(f"moe layer: {name} off by {err:.2e}")
        assert err < tol * 2.0 ** -8, name


def test_masked_tokens_leave_the_layer_alone():
    """NaN in a padding token's logits reaches neither the output nor a gradient."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, logits = torch.randn((12, 64), device="cuda", generator=gen).bfloat16(), torch.randn((12, 5), device="cuda", generator=gen)
    w = torch.randn((5, 64, 64), device="cuda", generator=gen).bfloat16()
    logits[[2, 7]] = float("nan")
    mask = torch.ones(12, dtype=torch.bool, device="cuda")
    mask[[2, 7]] = False
    layer = moe_layer.TrainingLayer(12, 2, w)
    log("moe layer: masked tokens")
    out = layer.forward(x, logits, mask)
    assert torch.isfinite(out).all() and (out[[2, 7]] == 0).all()
    for g in layer.backward(torch.randn((12, 64), device="cuda", generator=gen)):
        assert torch.isfinite(g).all()
    assert int(layer.ep.recv_token_per_expert.sum()) == 20
