"""A mixture-of-experts layer from the library's calls, for serving and for
training.

``ServingLayer`` is the whole int8 layer of one device: router, layout +
notify + dispatch (int8 rows), first expert matmul with its SwiGLU epilogue,
second expert matmul back to bf16 rows, combine.  Seven launches, every buffer
allocated once, nothing read by the host, so a step can be captured in a HIP
graph.

``TrainingLayer`` routes bf16 rows to linear experts (torch products) and
carries gradients back through the combine, the experts, the dispatch and the
router.

Run it to see both against plain torch:  python examples/moe_layer.py
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_moe_layout_03_amd as M  # noqa: E402


class ServingLayer:
    """w1 int8 [E, 2n, h] (gate rows, then up rows) with scales [E, 2n], w2 int8 [E, h, n] with scales [E, h], gate
    [E, h] and bias [E] of the router; up to ``tokens`` tokens a step, whose results stand in the first rows of
    ``idx``, ``weights`` and ``out``."""

    def __init__(self, tokens, topk, w1, w1_scale, w2, w2_scale, gate, bias, groups, topk_groups, scale):
        self.w1, self.w1_scale, self.w2, self.w2_scale = w1, w1_scale, w2, w2_scale
        self.gate, self.bias, self.groups, self.topk_groups, self.scale = gate, bias, groups, topk_groups, scale
        experts, hidden, n = w2.shape
        self.hidden, self.n, self.rows = hidden, n, tokens * topk
        dev = w1.device
        self.ep = M.EpBuffers(tokens, hidden, topk, experts, 1, device=dev)
        self.idx = torch.zeros((tokens, topk), dtype=torch.int32, device=dev)
        self.weights = torch.zeros((tokens, topk), device=dev)
        self.act_bytes = M.moe_recv_row_bytes(n, M.MOE_INT8_ROWSCALE)
        self.act = torch.zeros(self.rows * self.act_bytes, dtype=torch.uint8, device=dev)
        self.workspace = torch.zeros(M.moe_gemm_swiglu_quant_workspace_bytes(self.rows, n), dtype=torch.uint8,
                                     device=dev)
        self.out_rows = torch.zeros((self.rows, hidden), dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=dev)

    def step(self, x, token_mask=None):
        ep, bs = self.ep, x.shape[0]
        idx, weights, out = self.idx[:bs], self.weights[:bs], self.out[:bs]
        logits = x.float() @ self.gate.t()
        M.moe_route(logits, idx, weights, M.MOE_SCORE_SIGMOID, bias=self.bias, num_groups=self.groups,
                    topk_groups=self.topk_groups, group_top=2, scale=self.scale, token_mask=token_mask)
        ep.layout_notify_dispatch(x, idx)
        scale, stride = M.token_scales_of(ep.recv_x, self.hidden)
        M.moe_grouped_gemm_swiglu_quant_i8(ep.recv_x, ep.row_bytes, self.rows, self.hidden, ep.recv_token_per_expert,
                                           self.w1, self.w1_scale, scale, self.act, self.workspace, stride)
        scale, stride = M.token_scales_of(self.act, self.n)
        M.moe_grouped_gemm_deq_i8(self.act, self.act_bytes, self.rows, self.n, ep.recv_token_per_expert, self.w2,
                                  self.w2_scale, scale, self.out_rows, stride)
        M.moe_combine(self.out_rows, M.MOE_BF16, self.hidden, idx, weights, ep.send_token_idx, ep.put_offset,
                      ep.recv_base, ep.epr, ep.ranks, out)
        return out


class TrainingLayer:
    """Linear experts w bf16 [E, h, h] (y = x w^T) behind a softmax router."""

    def __init__(self, tokens, topk, w):
        self.w = w
        experts, self.hidden, _ = w.shape
        dev = w.device
        self.ep = M.EpBuffers(tokens, self.hidden, topk, experts, 1, quant_int8=False, out_dtype=torch.float32,
                              device=dev)
        self.idx = torch.zeros((tokens, topk), dtype=torch.int32, device=dev)
        self.weights = torch.zeros((tokens, topk), device=dev)
        self.ones = torch.ones((tokens, topk), device=dev)

    def _ranges(self):
        first = 0
        for e, count in enumerate(self.ep.recv_token_per_expert.tolist()):
            if count:
                yield e, slice(first, first + count)
            first += count

    def forward(self, x, logits, token_mask=None):
        ep = self.ep
        self.logits = logits
        M.moe_route(logits, self.idx, self.weights, M.MOE_SCORE_SOFTMAX, token_mask=token_mask)
        ep.layout_notify_dispatch(x, self.idx)
        self.x_rows = ep.recv_x.view(torch.bfloat16).view(-1, self.hidden)
        self.y_rows = torch.zeros_like(self.x_rows)
        for e, r in self._ranges():
            torch.mm(self.x_rows[r], self.w[e].t(), out=self.y_rows[r])
        M.moe_combine(self.y_rows, M.MOE_BF16, self.hidden, self.idx, self.weights, ep.send_token_idx, ep.put_offset,
                      ep.recv_base, ep.epr, ep.ranks, ep.out)
        return ep.out

    def backward(self, grad_out):
        """-> gradients of x (fp32), the logits and the experts' weights."""
        ep = self.ep
        grad_weights = torch.empty_like(self.weights)
        # in place: the rows that combine read become their gradients
        grad_y = self.y_rows
        M.moe_combine_backward(grad_out, self.y_rows, M.MOE_BF16, self.idx, self.weights, ep.send_token_idx,
                               ep.put_offset, ep.recv_base, ep.epr, ep.ranks, grad_y, grad_weights)
        grad_w, grad_x_rows = torch.zeros_like(self.w), torch.zeros_like(self.x_rows)
        for e, r in self._ranges():
            torch.mm(grad_y[r].t(), self.x_rows[r], out=grad_w[e])
            torch.mm(grad_y[r], self.w[e], out=grad_x_rows[r])
        grad_x = torch.empty_like(grad_out, dtype=torch.float32)
        M.moe_combine(grad_x_rows, M.MOE_BF16, self.hidden, self.idx, self.ones, ep.send_token_idx, ep.put_offset,
                      ep.recv_base, ep.epr, ep.ranks, grad_x)
        grad_logits = torch.empty_like(self.logits)
        M.moe_route_backward(grad_weights, self.logits, self.idx, M.MOE_SCORE_SOFTMAX, grad_logits)
        return grad_x, grad_logits, grad_w


def quantised(w):
    """int8 codes and a scale for each output channel (the last dimension is summed over)."""
    scale = w.abs().amax(dim=-1).clamp(min=1e-12) / 127
    return (w / scale[..., None]).round().clamp(-127, 127).to(torch.int8), scale.float().contiguous()


def serving_example(tokens=48, hidden=256, n=128, experts=16, topk=4, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x = rand(tokens, hidden).bfloat16()
    w1, w2 = rand(experts, 2 * n, hidden) / hidden ** 0.5, rand(experts, hidden, n) / n ** 0.5
    gate, bias = rand(experts, hidden) / hidden ** 0.5 * 2, rand(experts) * 0.05
    (q1, s1), (q2, s2) = quantised(w1), quantised(w2)
    layer = ServingLayer(tokens, topk, q1, s1, q2, s2, gate, bias, 4, 2, 2.5)
    mask = torch.ones(tokens, dtype=torch.uint8, device="cuda")
    mask[3] = 0
    out = layer.step(x, mask).double()
    # the same layer in 64 bits, without quantising
    y = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    for j in range(topk):
        for e in range(experts):
            at = layer.idx[:, j] == e
            h = x[at].double() @ w1[e].double().t()
            act = torch.nn.functional.silu(h[:, :n]) * h[:, n:]
            y[at] += layer.weights[at, j, None].double() * (act @ w2[e].double().t())
    return out, y, layer


def training_example(tokens=40, hidden=64, experts=6, topk=2, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x, logits = rand(tokens, hidden).bfloat16(), rand(tokens, experts)
    w, grad_out = (rand(experts, hidden, hidden) / hidden ** 0.5).bfloat16(), rand(tokens, hidden)
    layer = TrainingLayer(tokens, topk, w)
    out = layer.forward(x, logits)
    got = (out.clone(),) + layer.backward(grad_out)
    # autograd over the same choice in 64 bits
    xd, ld, wd = (t.double().requires_grad_() for t in (x, logits, w))
    idx = layer.idx.long()
    p = torch.softmax(torch.gather(ld, 1, idx), dim=1)
    rows = torch.matmul(wd[idx.reshape(-1)], xd.repeat_interleave(topk, 0)[:, :, None])[:, :, 0]
    ref = (rows.view(tokens, topk, hidden) * p[:, :, None]).sum(1)
    ref.backward(grad_out.double())
    return got, (ref.detach(), xd.grad, ld.grad, wd.grad)


def main():
    out, ref, _ = serving_example()
    print(f"serving: int8 layer against 64 bits, relative error {float((out - ref).norm() / ref.norm()):.4f}")
    names = ("output", "grad x", "grad logits", "grad w")
    for name, a, b in zip(names, *training_example()):
        print(f"training: {name}, relative error {float((a.double() - b).norm() / b.norm()):.5f}")


if __name__ == "__main__":
    main()
