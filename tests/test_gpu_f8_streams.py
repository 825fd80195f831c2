"""The norm, its gradient and the 8-bit float products on streams of their own at the same time, and the gradient in
place over batches that a workgroup walks."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log
from instance_cases_f8 import GATED, PLAIN
from test_gpu_gemm_f8 import inputs, on_device, workspace
from test_gpu_norm import check_backward, make

pytestmark = pytest.mark.gpu


class Products:
    """A plain and a gated product with buffers of their own."""

    def __init__(self, name, gated_name, seed, k=400):
        rng = np.random.default_rng(seed)
        self.k = k
        self.rows, n, counts = PLAIN[name]
        a, ts, w, ws = inputs(rng, self.rows, k, n, len(counts), 1)
        self.plain = on_device(a, ts, w, ws, counts)
        self.out = torch.zeros((self.rows, n), dtype=torch.bfloat16, device="cuda")
        self.gated_rows, n, counts = GATED[gated_name]
        a, ts, w, ws = inputs(rng, self.gated_rows, k, n, len(counts), 2)
        self.gated = on_device(a, ts, w, ws, counts)
        self.q = torch.zeros(self.gated_rows * B.row_bytes(n), dtype=torch.uint8, device="cuda")
        self.workspace = workspace(self.gated_rows, n)

    def step(self, stream):
        a, rb, scale, stride, w, ws, count = self.plain
        M.moe_grouped_gemm_f8(a, rb, self.rows, self.k, count, w, ws, scale, self.out, stride, stream=stream)
        a, rb, scale, stride, w, ws, count = self.gated
        M.moe_grouped_gemm_swiglu_quant_f8(a, rb, self.gated_rows, self.k, count, w, ws, scale, self.q, self.workspace,
                                           stride, stream=stream)

    def results(self):
        return [self.out, self.q]


class Norm:
    """A norm and its gradient."""

    def __init__(self, bs, h, seed):
        rng = np.random.default_rng(seed)
        self.x, self.r, self.g = (make(rng, bs, h, "bf16") for _ in range(3))
        self.w = torch.from_numpy((rng.random(h) + 0.5).astype(np.float32)).cuda()
        self.sum, self.out, self.dx = (torch.zeros_like(self.x) for _ in range(3))
        self.rows = torch.zeros(bs * B.row_bytes(h), dtype=torch.uint8, device="cuda")
        self.rstd, self.dw = torch.zeros(bs, device="cuda"), torch.zeros(h, device="cuda")
        self.workspace = torch.zeros(M.moe_rms_norm_backward_workspace_bytes(bs, h), dtype=torch.uint8, device="cuda")

    def step(self, stream):
        M.moe_rms_norm(self.x, self.w, 1e-6, residual=self.r, sum=self.sum, out=self.out, rows=self.rows, rstd=self.rstd,
                       stream=stream)
        M.moe_rms_norm_backward(self.g, self.sum, self.w, self.rstd, self.dx, grad_weight=self.dw,
                                workspace=self.workspace, stream=stream)

    def results(self):
        return [self.sum, self.out, self.rows, self.rstd, self.dx, self.dw]


def test_streams_at_the_same_time():
    """Four streams, several rounds: each gives what it gives alone, bit for bit."""
    work = [Products("split16", "tile64", 1), Products("tile256", "split16", 2), Products("tile64", "whole", 3),
            Norm(1500, 1040, 4)]
    alone = []
    for w in work:
        log(f"8-bit float path alone {type(w).__name__}")
        w.step(None)
        torch.cuda.synchronize()
        alone.append([r.clone() for r in w.results()])
    streams = [torch.cuda.Stream() for _ in work]
    for turn in range(3):
        for w in work:
            for r in w.results():
                r.zero_()
        torch.cuda.synchronize()
        log(f"8-bit float path on four streams, turn {turn}")
        for _ in range(4):
            for w, s in zip(work, streams):
                w.step(s)
        torch.cuda.synchronize()
        for w, want in zip(work, alone):
            assert all(torch.equal(a, b) for a, b in zip(w.results(), want))


@pytest.mark.parametrize("bs,h", [(2100, 72), (1030, 1032), (600, 4104), (600, 8200)])
def test_gradient_in_place_over_many_rows(bs, h):
    """More rows than workgroups hold at once: the next rows are loaded before these are stored."""
    rng = np.random.default_rng(h)
    check_backward(rng, bs, h, "bf16", in_place="skip")
    check_backward(rng, bs, h, "bf16", "bf16", in_place="grad")
    check_backward(rng, bs, h, "fp32", "fp32", skip=False, mask=rng.random(bs) < 0.6, in_place="grad")
