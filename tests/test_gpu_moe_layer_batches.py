"""The example's serving layer with fewer tokens than it was made for."""

import os
import sys

import pytest
import torch

from gpu_util import log

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def test_fewer_tokens_a_step():
    """A batch gives what a layer made for just that batch gives, bit for bit, and the rest of the outputs stays."""
    _, _, layer = moe_layer.serving_example(tokens=40, seed=2)
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((40, layer.hidden), device="cuda", generator=gen).bfloat16()
    topk = layer.idx.shape[1]
    for bs in (1, 7, 39, 0, 40):
        log(f"moe layer: {bs} of 40 tokens")
        own = moe_layer.ServingLayer(max(bs, 1), topk, layer.w1, layer.w1_scale, layer.w2, layer.w2_scale, layer.gate,
                                     layer.bias, layer.groups, layer.topk_groups, layer.scale)
        mask = torch.ones(bs, dtype=torch.uint8, device="cuda") if bs % 2 else None
        for t in (layer.out, layer.weights, layer.idx):
            t.fill_(7)
        got = layer.step(x[:bs].contiguous(), mask)
        torch.cuda.synchronize()
        assert got.shape == (bs, layer.hidden)
        assert all((t[bs:] == 7).all() for t in (layer.out, layer.weights, layer.idx))
        if bs > 0:
            want = own.step(x[:bs].contiguous(), mask)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
            assert torch.equal(layer.idx[:bs], own.idx) and torch.equal(layer.weights[:bs], own.weights)
            assert int(layer.ep.recv_token_per_expert.sum()) == bs * topk
