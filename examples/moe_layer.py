"""A mixture-of-experts layer from the library's calls, for serving and for
training.

``ServingLayer`` is the whole int8 layer of one device: router, layout +
notify + dispatch (int8 rows), first expert matmul with its SwiGLU epilogue,
second expert matmul back to bf16 rows, combine.  Seven launches, every buffer
allocated once, nothing read by the host, so a step can be captured in a HIP
graph.

``Float8Layer`` is the same layer in 8-bit floats with what stands in front of
it: residual addition and norm (whose e4m3 rows are dispatched as they are),
router, dispatch, both expert products, combine.

``TrainingLayer`` routes bf16 rows to linear experts (torch products) and
carries gradients back through the combine, the experts, the dispatch and the
router.

``NormedTrainingLayer`` is that one behind a norm with a residual, whose
gradients it carries on.

Run it to see them against plain torch:  python examples/moe_layer.py
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


class Float8Layer:
    """norm_weight float [h]; w1 e4m3 [E, 2n, h] (gate rows, then up rows) with scales [E, 2 blocks of n, blocks of h],
    w2 e4m3 [E, h, n] with scales [E, blocks of h, blocks of n]; gate, bias and the rest as ``ServingLayer``.  A step
    takes the layer's input and the residual stream; the sum of both stands in ``sum``, the stream for the next layer,
    to which ``out`` is the next input."""

    def __init__(self, tokens, topk, norm_weight, w1, w1_scale, w2, w2_scale, gate, bias, groups, topk_groups, scale):
        self.norm_weight, self.w1, self.w1_scale, self.w2, self.w2_scale = norm_weight, w1, w1_scale, w2, w2_scale
        self.gate, self.bias, self.groups, self.topk_groups, self.scale = gate, bias, groups, topk_groups, scale
        experts, hidden, n = w2.shape
        self.hidden, self.n, self.rows = hidden, n, tokens * topk
        dev = w1.device
        self.ep = M.EpBuffers(tokens, hidden, topk, experts, 1, x_dtype=torch.float8_e4m3fn, quant_int8=False,
                              device=dev)
        self.idx = torch.zeros((tokens, topk), dtype=torch.int32, device=dev)
        self.weights = torch.zeros((tokens, topk), device=dev)
        self.sum, self.normed, self.out = (torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=dev)
                                           for _ in range(3))
        self.token_rows = torch.zeros((tokens, self.ep.row_bytes), dtype=torch.uint8, device=dev)
        self.act_bytes = M.moe_recv_row_bytes(n, M.MOE_E4M3_BLOCKSCALE)
        self.act = torch.zeros(self.rows * self.act_bytes, dtype=torch.uint8, device=dev)
        self.workspace = torch.zeros(M.moe_gemm_swiglu_quant_f8_workspace_bytes(self.rows, n), dtype=torch.uint8,
                                     device=dev)
        self.out_rows = torch.zeros((self.rows, hidden), dtype=torch.bfloat16, device=dev)

    def step(self, x, residual, token_mask=None):
        ep, bs = self.ep, x.shape[0]
        idx, weights, normed, out = self.idx[:bs], self.weights[:bs], self.normed[:bs], self.out[:bs]
        M.moe_rms_norm(x, self.norm_weight, 1e-6, residual=residual, sum=self.sum[:bs], out=normed,
                       rows=self.token_rows[:bs])
        logits = normed.float() @ self.gate.t()
        M.moe_route(logits, idx, weights, M.MOE_SCORE_SIGMOID, bias=self.bias, num_groups=self.groups,
                    topk_groups=self.topk_groups, group_top=2, scale=self.scale, token_mask=token_mask)
        ep.layout_notify_dispatch(self.token_rows[:bs], idx)
        scale, stride = M.block_scales_of(ep.recv_x, self.hidden)
        M.moe_grouped_gemm_swiglu_quant_f8(ep.recv_x, ep.row_bytes, self.rows, self.hidden, ep.recv_token_per_expert,
                                           self.w1, self.w1_scale, scale, self.act, self.workspace, stride)
        scale, stride = M.block_scales_of(self.act, self.n)
        M.moe_grouped_gemm_f8(self.act, self.act_bytes, self.rows, self.n, ep.recv_token_per_expert, self.w2,
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


class NormedTrainingLayer:
    """``TrainingLayer`` behind a norm: forward(x, residual, logits) -> (the layer's output, the residual stream)."""

    def __init__(self, tokens, topk, w, norm_weight):
        self.layer, self.norm_weight = TrainingLayer(tokens, topk, w), norm_weight
        hidden, dev = w.shape[1], w.device
        self.sum, self.normed = (torch.zeros((tokens, hidden), dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.rstd = torch.zeros(tokens, device=dev)
        self.workspace = torch.zeros(M.moe_rms_norm_backward_workspace_bytes(tokens, hidden), dtype=torch.uint8,
                                     device=dev)

    def forward(self, x, residual, logits, token_mask=None):
        M.moe_rms_norm(x, self.norm_weight, 1e-6, residual=residual, sum=self.sum, out=self.normed, rstd=self.rstd)
        self.token_mask = token_mask
        return self.layer.forward(self.normed, logits, token_mask), self.sum

    def backward(self, grad_out, grad_stream):
        """-> gradients of x (and, the same, of the residual), the norm's weight, the logits, the experts' weights."""
        grad_normed, grad_logits, grad_w = self.layer.backward(grad_out)
        grad_x, grad_norm = torch.empty_like(self.sum), torch.empty_like(self.norm_weight)
        M.moe_rms_norm_backward(grad_normed, self.sum, self.norm_weight, self.rstd, grad_x, grad_sum=grad_stream,
                                grad_weight=grad_norm, workspace=self.workspace, token_mask=self.token_mask)
        return grad_x, grad_norm, grad_logits, grad_w


def quantised_blocks(w):
    """e4m3 codes of w [E, n, k] and a scale for each block of 128 x 128."""
    e, n, k = w.shape
    padded = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128))
    blocks = padded.view(e, padded.shape[1] // 128, 128, padded.shape[2] // 128, 128)
    scale = blocks.abs().amax(dim=(2, 4)).clamp(min=1e-12) / 448
    codes = (blocks / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).view(padded.shape)
    return codes[:, :n, :k].contiguous(), scale.float().contiguous()


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


def float8_example(tokens=48, hidden=256, n=160, experts=16, topk=4, seed=2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x, residual = rand(tokens, hidden).bfloat16(), (rand(tokens, hidden) * 2).bfloat16()
    w1, w2 = rand(experts, 2 * n, hidden) / hidden ** 0.5, rand(experts, hidden, n) / n ** 0.5
    gate, bias = rand(experts, hidden) / hidden ** 0.5 * 2, rand(experts) * 0.05
    norm_weight = 0.5 + torch.rand(hidden, device="cuda", generator=gen)
    gate_codes, gate_scale = quantised_blocks(w1[:, :n])
    up_codes, up_scale = quantised_blocks(w1[:, n:])
    q1, s1 = torch.cat([gate_codes, up_codes], dim=1), torch.cat([gate_scale, up_scale], dim=1)
    q2, s2 = quantised_blocks(w2)
    layer = Float8Layer(tokens, topk, norm_weight, q1, s1, q2, s2, gate, bias, 4, 2, 2.5)
    mask = torch.ones(tokens, dtype=torch.uint8, device="cuda")
    mask[3] = 0
    out = layer.step(x, residual, mask).double()
    # the same layer in 64 bits, without quantising
    s = x.double() + residual.double()
    h = s / (s.square().mean(dim=1, keepdim=True) + 1e-6).sqrt() * norm_weight.double()
    y = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
    for j in range(topk):
        for e in range(experts):
            at = layer.idx[:, j] == e
            u = h[at] @ w1[e].double().t()
            act = torch.nn.functional.silu(u[:, :n]) * u[:, n:]
            y[at] += layer.weights[at, j, None].double() * (act @ w2[e].double().t())
    return out, y, layer


def normed_training_example(tokens=40, hidden=64, experts=6, topk=2, seed=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    x, residual, logits = rand(tokens, hidden).bfloat16(), rand(tokens, hidden).bfloat16(), rand(tokens, experts)
    w, grad_out = (rand(experts, hidden, hidden) / hidden ** 0.5).bfloat16(), rand(tokens, hidden)
    norm_weight, grad_stream = 0.5 + torch.rand(hidden, device="cuda", generator=gen), rand(tokens, hidden).bfloat16()
    layer = NormedTrainingLayer(tokens, topk, w, norm_weight)
    out, stream = layer.forward(x, residual, logits)
    got = (out.clone(), stream.clone()) + layer.backward(grad_out, grad_stream)
    # autograd over the same choice in 64 bits
    xd, nd, ld, wd = (t.double().requires_grad_() for t in (x, norm_weight, logits, w))
    s = xd + residual.double()
    h = s / (s.square().mean(dim=1, keepdim=True) + 1e-6).sqrt() * nd
    idx = layer.layer.idx.long()
    p = torch.softmax(torch.gather(ld, 1, idx), dim=1)
    rows = torch.matmul(wd[idx.reshape(-1)], h.repeat_interleave(topk, 0)[:, :, None])[:, :, 0]
    ref = (rows.view(tokens, topk, hidden) * p[:, :, None]).sum(1)
    torch.autograd.backward((ref, s), (grad_out.double(), grad_stream.double()))
    return got, (ref.detach(), s.detach(), xd.grad, nd.grad, ld.grad, wd.grad)


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
    out, ref, _ = float8_example()
    print(f"serving: 8-bit float layer against 64 bits, relative error {float((out - ref).norm() / ref.norm()):.4f}")
    names = ("output", "stream", "grad x", "grad norm weight", "grad logits", "grad w")
    for name, a, b in zip(names, *normed_training_example()):
        print(f"training behind a norm: {name}, relative error {float((a.double() - b).norm() / b.norm()):.5f}")
    names = ("output", "grad x", "grad logits", "grad w")
    for name, a, b in zip(names, *training_example()):
        print(f"training: {name}, relative error {float((a.double() - b).norm() / b.norm()):.5f}")


if __name__ == "__main__":
    main()
