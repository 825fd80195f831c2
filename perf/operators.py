"""The router, its gradient, the combine's gradient and the second expert
product as measured cases: inputs, the plain form of each operator in
elementary torch operations, the library's calls, and the operators'
definitions in 64 bits.

Four operators (``case["op"]``):

route           scores of the experts, biased and grouped choice of the top k,
                renormalised weights
route_backward  the gradient of the weights carried back to the logits
combine_backward  the gradient of the weighted sum of a token's rows: the
                rows' gradients and the weights'
gemm_deq        int8 receive rows times their expert's int8 weights, scaled by
                token and by channel, rounded to the row type combine reads
"""

import math
import types

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_GRID = 2.0 ** 30   # selection values with a bias are compared on this grid
_CLIP = 1024.0      # and within these bounds


def listed():
    return [
        # one token of a decode step: 256 experts in 8 groups, the best 4 kept
        dict(name="route_decode", op="route", bs=1, experts=256, topk=8, type="fp32", score="sigmoid", bias=True,
             groups=8, keep=4, group_top=2, renorm=True, scale=2.5, masked=0.0),
        # a prefill of the same router
        dict(name="route_prefill", op="route", bs=16384, experts=256, topk=8, type="fp32", score="sigmoid", bias=True,
             groups=8, keep=4, group_top=2, renorm=True, scale=2.5, masked=0.0),
        # a training batch of a softmax router, logits in bf16, padding tokens masked, an odd batch
        dict(name="route_softmax", op="route", bs=4095, experts=64, topk=6, type="bf16", score="softmax", bias=False,
             groups=1, keep=1, group_top=1, renorm=False, scale=1.0, masked=0.05),
        # the training step's gradient of the large grouped router
        dict(name="route_backward_large", op="route_backward", bs=16384, experts=256, topk=8, type="fp32",
             score="sigmoid", renorm=True, scale=2.5, masked=0.0),
        # the softmax router's gradient reaches every expert's logit
        dict(name="route_backward_softmax", op="route_backward", bs=4095, experts=64, topk=6, type="bf16",
             score="softmax", renorm=False, scale=1.0, masked=0.05),
        # a training step's combine at the library's large shape
        dict(name="combine_backward_large", op="combine_backward", bs=4096, hidden=7168, topk=8, experts=256, ranks=16,
             type="bf16", grad="bf16", masked=0.0),
        # a ragged micro-batch with padding tokens, gradients in fp32
        dict(name="combine_backward_small", op="combine_backward", bs=61, hidden=1000, topk=5, experts=24, ranks=3,
             type="fp16", grad="fp32", masked=0.1),
        # one rank's share of a decode step: a row or two for each of its experts
        dict(name="gemm_deq_decode", op="gemm_deq", rows=24, k=2048, n=7168, groups=16, skew=0.5, type="bf16"),
        # a step of many sequences: tens of rows for each expert
        dict(name="gemm_deq_batch", op="gemm_deq", rows=1000, k=2048, n=7168, groups=16, skew=0.5, type="bf16"),
        # one rank's share of a prefill: thousands of rows for each expert
        dict(name="gemm_deq_prefill", op="gemm_deq", rows=32768, k=2048, n=7168, groups=16, skew=0.3, type="bf16"),
        # ragged sizes, experts without rows
        dict(name="gemm_deq_ragged", op="gemm_deq", rows=777, k=1040, n=1001, groups=7, skew=2.0, type="fp16"),
        # a single row and a single expert: latency alone
        dict(name="gemm_deq_single", op="gemm_deq", rows=1, k=512, n=1024, groups=1, skew=0.0, type="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "combine_backward", "gemm_deq", "gemm_deq"])
    masked = rng.choice([0.0, 0.0, 0.05, 0.3])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        keep = rng.randint(1, groups)
        group_top = rng.choice([1, 2])
        score = rng.choice(["softmax", "sigmoid"])
        case = dict(op=op, bs=_log(rng, 1, max(2, min(16384, 4_000_000 // experts))), experts=experts,
                    topk=rng.randint(1, min(keep * (experts // groups), 16)), type=rng.choice(["bf16", "fp16", "fp32"]),
                    score=score, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 0.3]), masked=masked)
        if op == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, keep=keep, group_top=group_top)
        return case
    if op == "combine_backward":
        topk = rng.randint(1, 12)
        hidden = 8 * _log(rng, 8, 1024)
        ranks = rng.choice([1, 2, 4, 8])
        experts = ranks * rng.randint((topk + ranks - 1) // ranks, 32)
        bs = _log(rng, 1, max(2, min(4096, 200_000_000 // (hidden * topk))))
        return dict(op=op, bs=bs, hidden=hidden, topk=topk, experts=experts, ranks=ranks,
                    type=rng.choice(["bf16", "fp16"]), grad=rng.choice(["bf16", "fp16", "fp32"]), masked=masked)
    k, n = 16 * _log(rng, 4, 448), _log(rng, 16, 8192)
    groups = _log(rng, 1, max(2, min(64, 230_000_000 // (k * n))))
    rows = _log(rng, 1, max(2, min(16384, 400_000_000_000 // (k * n))))
    return dict(op="gemm_deq", rows=rows, k=k, n=n, groups=groups, skew=rng.choice([0.0, 0.5, 1.0, 2.0]),
                type=rng.choice(["bf16", "fp16", "fp32"]))


def _counts(rows, groups, skew):
    """Rows of each expert: shares that fall with the expert's rank as rank^-skew, rounded by largest remainder."""
    share = np.arange(1, groups + 1, dtype=np.float64) ** -skew
    share *= rows / share.sum()
    got = np.floor(share).astype(np.int64)
    for i in np.argsort(got - share, kind="stable")[: rows - int(got.sum())]:
        got[i] += 1
    return got


def _row_bytes(width):
    """Bytes of an int8 receive row: codes, then the float scale at the next multiple of 32, in whole 128-byte lines."""
    return ((width + 31) // 32 * 32 + 32 + 127) // 128 * 128


def _logits(case, gen):
    bs, e = case["bs"], case["experts"]
    x = torch.randn((bs, e), generator=gen, device="cuda") * 1.5
    x = x + torch.randn((1, e), generator=gen, device="cuda") * 0.5  # some experts are liked more
    x = x.to(_TYPES[case["type"]])
    keep = torch.rand((bs,), generator=gen, device="cuda") >= case["masked"]
    x[~keep] = float("nan")  # what stands in padding tokens is anything
    return x, keep.to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = types.SimpleNamespace(case=dict(case))
    if case["op"] in ("route", "route_backward"):
        s.logits, s.mask = _logits(case, gen)
        bs, e, k = case["bs"], case["experts"], case["topk"]
        if case["op"] == "route":
            s.bias = torch.randn((e,), generator=gen, device="cuda") * 0.05 if case["bias"] else None
            s.idx = torch.zeros((bs, k), dtype=torch.int32, device="cuda")
            s.weights = torch.zeros((bs, k), dtype=torch.float32, device="cuda")
            return s
        # the choice that the forward pass made, and the gradient of its weights
        order = torch.sort(torch.nan_to_num(s.logits.float()), dim=1, descending=True, stable=True).indices[:, :k]
        s.idx = torch.where(s.mask[:, None] != 0, order, -1).to(torch.int32).contiguous()
        s.grad_weights = torch.randn((bs, k), generator=gen, device="cuda")
        s.grad_logits = torch.zeros_like(s.logits)
        return s
    if case["op"] == "combine_backward":
        bs, h, k, e, ranks = case["bs"], case["hidden"], case["topk"], case["experts"], case["ranks"]
        epr = e // ranks
        ids = torch.rand((bs, e), generator=gen, device="cuda").argsort(dim=1)[:, :k]
        keep = torch.rand((bs,), generator=gen, device="cuda") >= case["masked"]
        ids = torch.where(keep[:, None], ids, -1)
        flat = torch.where(ids < 0, e, ids).reshape(-1)
        order = torch.argsort(flat, stable=True)
        count = torch.bincount(flat, minlength=e + 1)
        start = count.cumsum(0) - count
        slot = torch.empty_like(flat)
        slot[order] = torch.arange(flat.numel(), device="cuda") - start[flat[order]]
        s.idx = ids.to(torch.int32)
        s.slot = torch.where(ids < 0, -1, slot.view(bs, k)).to(torch.int32)
        s.recv_base = start[:e:epr].to(torch.int32).contiguous()
        s.put_offset = (start[:e] - start[:e:epr].repeat_interleave(epr)).to(torch.int32)
        s.weights = torch.rand((bs, k), generator=gen, device="cuda") * (2.5 / k)
        s.recv = torch.randn((bs * k, h), generator=gen, device="cuda").to(_TYPES[case["type"]])
        s.grad_out = torch.randn((bs, h), generator=gen, device="cuda").to(_TYPES[case["grad"]])
        s.grad_recv = torch.zeros_like(s.recv)
        s.grad_weights = torch.zeros((bs, k), dtype=torch.float32, device="cuda")
        return s
    rows, k, n, groups = case["rows"], case["k"], case["n"], case["groups"]
    count = torch.from_numpy(_counts(rows, groups, case["skew"])).cuda()
    s.count = count[torch.rand((groups,), generator=gen, device="cuda").argsort()].to(torch.int32)
    s.most = int(_counts(rows, groups, case["skew"]).max())  # the plain form pads every expert to this
    s.row_bytes = _row_bytes(k)
    s.a = torch.zeros((rows, s.row_bytes), dtype=torch.uint8, device="cuda")
    s.a[:, :k] = _codes((rows, k), gen).view(torch.uint8)
    scale_at = (k + 31) // 32 * 32
    scale = (0.2 + torch.rand((rows, 1), generator=gen, device="cuda")) / 64
    s.a[:, scale_at:scale_at + 4] = scale.view(torch.uint8)
    s.a, s.scale_at = s.a.reshape(-1), scale_at
    s.w = _codes((groups, n, k), gen)
    s.w_scale = (0.2 + torch.rand((groups, n), generator=gen, device="cuda")) * (1.0 / (32 * math.sqrt(k)))
    s.out = torch.zeros((rows, n), dtype=_TYPES[case["type"]], device="cuda")
    return s


def _codes(shape, gen):
    """int8 codes as quantising a row of activations or weights leaves them."""
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in codes.view(-1).split(1 << 27):
        part.copy_((torch.randn(part.shape, generator=gen, device="cuda") * 36).round_().clamp_(-127, 127))
    return codes


# ---- the plain forms -----------------------------------------------------------


def _eligible(logits, mask):
    x = logits.float()
    ok = (x > -math.inf) & (mask[:, None] != 0)
    x = torch.where(ok, x.clamp(max=torch.finfo(torch.float32).max), 0.0)
    return x, ok


def _scores(x, ok, score):
    """Scores in 64 bits: the choice compares values that may stand next to each other."""
    d = x.double()
    if score == "sigmoid":
        return torch.where(ok, 1.0 / (1.0 + torch.exp(-d)), 0.0)
    top = torch.where(ok, d, -math.inf).amax(dim=1, keepdim=True)
    e = torch.where(ok, torch.exp(d - torch.where(top > -math.inf, top, 0.0)), 0.0)
    z = e.sum(dim=1, keepdim=True)
    return e / torch.where(z > 0, z, 1.0)


def _plain_route(s):
    c = s.case
    x, ok = _eligible(s.logits, s.mask)
    p = _scores(x, ok, c["score"])
    u = p if s.bias is None else p + s.bias.double()
    u = torch.where(ok, (torch.round(u * _GRID) / _GRID).clamp(-_CLIP, _CLIP), -math.inf)
    v = u if s.bias is not None else torch.where(ok, x.double(), -math.inf)
    if c["groups"] > 1:
        bs, size = x.shape[0], c["experts"] // c["groups"]
        if c["group_top"] == 1:
            g = v.view(bs, c["groups"], size).amax(dim=2)
        else:
            two = torch.sort(u.view(bs, c["groups"], size), dim=2, descending=True).values[:, :, :2]
            g = torch.where(two > -math.inf, two, 0.0).sum(dim=2)
            g = torch.where(two[:, :, 0] > -math.inf, g, -math.inf)
        best = torch.sort(g, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros_like(g, dtype=torch.bool).scatter_(1, best, True)
        v = torch.where(kept.repeat_interleave(size, dim=1), v, -math.inf)
    top = torch.sort(v, dim=1, descending=True, stable=True)
    at, found = top.indices[:, :c["topk"]], top.values[:, :c["topk"]] > -math.inf
    if c["renorm"]:
        d = torch.gather(x, 1, at).double()
        m = torch.where(found, d, -math.inf).amax(dim=1, keepdim=True)
        m = torch.where(found.any(dim=1, keepdim=True), m, 0.0)
        if c["score"] == "sigmoid":  # both parts of the ratio over e^min(m, 0)
            t = torch.exp(d - m.clamp(max=0.0)) / (1.0 + torch.exp(d))
            t = torch.where(d > 0, 1.0 / (1.0 + torch.exp(-d)) * torch.exp(-m.clamp(max=0.0)), t)
        else:
            t = torch.exp(d - m)
        t = torch.where(found, t, 0.0)
        z = t.sum(dim=1, keepdim=True)
        w = t / torch.where(z > 0, z, 1.0) * c["scale"]
    else:
        w = torch.where(found, torch.gather(p, 1, at), 0.0) * c["scale"]
    return torch.where(found, at, -1).to(torch.int32), w.float()


def _plain_route_backward(s):
    c = s.case
    chosen = s.idx >= 0
    x, ok = _eligible(s.logits, torch.ones_like(s.mask))
    at = torch.where(chosen, s.idx, 0).long()
    p = _scores(x, ok, c["score"])
    ps = torch.where(chosen, torch.gather(p, 1, at), 0.0)
    g = s.grad_weights.double() * c["scale"]
    if c["renorm"]:
        z = ps.sum(dim=1, keepdim=True)
        share = ps / torch.where(z > 0, z, 1.0)
        # d/dx of share_i through s_j, times s_j: the softmax of the chosen logits, or the sigmoid's with its slope
        ds = share * (g - (g * share).sum(dim=1, keepdim=True))
        if c["score"] == "sigmoid":
            ds = ds * (1.0 - ps)
        dx = torch.zeros_like(p).scatter_add_(1, at, torch.where(chosen, ds, 0.0))
    elif c["score"] == "sigmoid":
        dx = torch.zeros_like(p).scatter_add_(1, at, torch.where(chosen, g * ps * (1.0 - ps), 0.0))
    else:
        dx = torch.zeros_like(p).scatter_add_(1, at, torch.where(chosen, g * ps, 0.0))
        dx = dx - p * torch.where(chosen, g * ps, 0.0).sum(dim=1, keepdim=True)
    return dx.to(s.logits.dtype)


def _plain_combine_backward(s):
    c = s.case
    bs, h, k = c["bs"], c["hidden"], c["topk"]
    epr = c["experts"] // c["ranks"]
    good = s.idx >= 0
    e = torch.where(good, s.idx, 0).long()
    row = torch.where(good, s.recv_base[e // epr] + s.put_offset[e] + s.slot, bs * k).long()
    g = s.grad_out.float()
    y = torch.cat([s.recv, s.recv.new_zeros((1, h))]).float()[row.reshape(-1)].view(bs, k, h)
    grad_weights = (y * g[:, None, :]).sum(dim=2)
    grad_recv = s.recv.new_zeros((bs * k + 1, h))
    grad_recv[row.reshape(-1)] = (s.weights[:, :, None] * g[:, None, :]).to(s.recv.dtype).view(bs * k, h)
    return grad_recv[:bs * k], torch.where(good, grad_weights, 0.0)


def _plain_gemm_deq(s):
    c = s.case
    rows, k, groups = c["rows"], c["k"], c["groups"]
    a = s.a.view(rows, s.row_bytes)
    scale = a[:, s.scale_at:s.scale_at + 4].contiguous().view(torch.float32)
    end = s.count.long().cumsum(0)
    r = torch.arange(rows, device=s.a.device)
    g = torch.searchsorted(end, r, right=True)
    at = r - (end - s.count)[g]
    padded = torch.zeros((groups, s.most, k), dtype=torch.float32, device=s.a.device)
    padded[g, at] = a[:, :k].view(torch.int8).float()
    acc = torch.bmm(s.w.float(), padded.transpose(1, 2).contiguous())
    return ((acc.transpose(1, 2)[g, at] * s.w_scale[g]) * scale).to(s.out.dtype)


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "combine_backward": _plain_combine_backward,
          "gemm_deq": _plain_gemm_deq}


# ---- the library's calls -------------------------------------------------------


def _own(s):
    import combine_moe_layout_03_amd as M

    c = s.case
    if c["op"] == "gemm_deq":
        M.moe_grouped_gemm_deq_i8(s.a, s.row_bytes, c["rows"], c["k"], s.count, s.w, s.w_scale, s.a[s.scale_at:], s.out,
                                  token_scale_stride=s.row_bytes)
        return s.out
    if c["op"] == "combine_backward":
        rt = M.dtype_code(s.recv.dtype)
        M.moe_combine_backward(s.grad_out, s.recv, rt, s.idx, s.weights, s.slot, s.put_offset, s.recv_base,
                               c["experts"] // c["ranks"], c["ranks"], s.grad_recv, s.grad_weights)
        return s.grad_recv, s.grad_weights
    score = M.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else M.MOE_SCORE_SOFTMAX
    if c["op"] == "route":
        M.moe_route(s.logits, s.idx, s.weights, score, bias=s.bias, num_groups=c["groups"], topk_groups=c["keep"],
                    group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"], token_mask=s.mask)
        return s.idx, s.weights
    M.moe_route_backward(s.grad_weights, s.logits, s.idx, score, s.grad_logits, renormalize=c["renorm"],
                         scale=c["scale"])
    return s.grad_logits


def run(state):
    return _own(state) if own else _PLAIN[state.case["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------


def work(case):
    op = case["op"]
    if op in ("route", "route_backward"):
        bs, e, k, es = case["bs"], case["experts"], case["topk"], _BYTES[case["type"]]
        if op == "route":
            return {"bytes": bs * (e * es + 8 * k + 1) + (4 * e if case["bias"] else 0), "flops": 4 * bs * e}
        return {"bytes": bs * (2 * e * es + 8 * k), "flops": 4 * bs * e}
    if op == "combine_backward":
        bs, h, k = case["bs"], case["hidden"], case["topk"]
        rows = bs * k * (1.0 - case["masked"])
        return {"bytes": bs * h * _BYTES[case["grad"]] + 4 * rows * h + 16 * bs * k, "flops": 3 * rows * h}
    rows, k, n = case["rows"], case["k"], case["n"]
    active = int((_counts(rows, case["groups"], case["skew"]) > 0).sum())
    return {"bytes": rows * (k + 4) + active * n * (k + 4) + rows * n * _BYTES[case["type"]], "flops": 2 * rows * n * k}


# ---- the definitions in 64 bits ------------------------------------------------


def _np(t):
    return t.detach().double().cpu().numpy()


def _np_scores(x, ok, score):
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            return np.where(ok, 1 / (1 + np.exp(-x)), 0)
        m = np.max(np.where(ok, x, -np.inf), axis=1, keepdims=True)
        e = np.where(ok, np.exp(x - np.where(np.isfinite(m), m, 0)), 0)
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)


def _exact_route(s):
    c = s.case
    x = _np(s.logits)
    ok = (np.nan_to_num(x, nan=-np.inf) > -np.inf) & (_np(s.mask)[:, None] > 0)
    x = np.where(ok, np.minimum(x, np.finfo(np.float32).max), 0)
    p = _np_scores(x, ok, c["score"])
    u = np.clip(np.rint((p + (_np(s.bias) if s.bias is not None else 0)) * _GRID) / _GRID, -_CLIP, _CLIP)
    v = np.where(ok, u if s.bias is not None else x, -np.inf)
    if c["groups"] > 1:
        bs = x.shape[0]
        if c["group_top"] == 1:
            g = v.reshape(bs, c["groups"], -1).max(axis=2)
        else:
            two = -np.sort(-np.where(ok, u, -np.inf).reshape(bs, c["groups"], -1), axis=2)[:, :, :2]
            g = np.where(np.isfinite(two[:, :, 0]), np.where(np.isfinite(two), two, 0).sum(axis=2), -np.inf)
        rank = np.argsort(np.argsort(-g, axis=1, kind="stable"), axis=1, kind="stable")
        v = np.where(np.repeat(rank < c["keep"], c["experts"] // c["groups"], axis=1), v, -np.inf)
    at = np.argsort(-v, axis=1, kind="stable")[:, :c["topk"]]
    found = np.isfinite(np.take_along_axis(v, at, axis=1))
    w = np.where(found, np.take_along_axis(p, at, axis=1), 0)
    if c["renorm"]:
        w = w / np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
    return np.where(found, at, -1).astype(np.int32), w * c["scale"]


def _exact_route_backward(s):
    """The chain rule with each step's Jacobian as a matrix product over the chosen entries."""
    c = s.case
    x = _np(s.logits)
    idx = s.idx.cpu().numpy().astype(np.int64)
    chosen = idx >= 0
    ok = np.nan_to_num(x, nan=-np.inf) > -np.inf
    p = _np_scores(np.where(ok, x, 0), ok, c["score"])
    at = np.where(chosen, idx, 0)
    ps = np.where(chosen, np.take_along_axis(p, at, axis=1), 0)
    g = np.where(chosen, _np(s.grad_weights), 0) * c["scale"]
    if c["renorm"]:  # w = s / Z: dL/ds_j = g_j / Z - sum_i g_i s_i / Z^2
        z = np.where(chosen.any(axis=1, keepdims=True), ps.sum(axis=1, keepdims=True), 1)
        ds = np.where(chosen, g / z - (g * ps).sum(axis=1, keepdims=True) / z ** 2, 0)
    else:
        ds = g
    full = np.zeros_like(p)
    rows = np.broadcast_to(np.arange(x.shape[0])[:, None], at.shape)
    np.add.at(full, (rows[chosen], at[chosen]), ds[chosen])
    if c["score"] == "sigmoid":
        return full * p * (1 - p)
    return p * (full - (full * p).sum(axis=1, keepdims=True))


def _exact_combine_backward(s):
    c = s.case
    epr = c["experts"] // c["ranks"]
    g = s.grad_out.double()
    grad_recv = torch.zeros(s.recv.shape, dtype=torch.float64, device=s.recv.device)
    grad_weights = torch.zeros(s.weights.shape, dtype=torch.float64, device=s.recv.device)
    for j in range(c["topk"]):
        t = torch.nonzero(s.idx[:, j] >= 0).reshape(-1)
        e = s.idx[t, j].long()
        row = (s.recv_base[e // epr] + s.put_offset[e] + s.slot[t, j]).long()
        grad_recv[row] = s.weights[t, j].double()[:, None] * g[t]
        grad_weights[t, j] = torch.linalg.vecdot(s.recv[row].double(), g[t])
    return grad_recv, grad_weights


def _exact_gemm_deq(s):
    c = s.case
    rows, k = c["rows"], c["k"]
    a = s.a.view(rows, s.row_bytes)
    scale = a[:, s.scale_at:s.scale_at + 4].contiguous().view(torch.float32).double()
    out = torch.zeros((rows, c["n"]), dtype=torch.float64, device=s.a.device)
    first = 0
    for g, count in enumerate(s.count.tolist()):
        part = slice(first, first + count)
        acc = a[part, :k].contiguous().view(torch.int8).double() @ s.w[g].double().t()
        out[part] = acc * s.w_scale[g].double() * scale[part]
        first += count
    return out


_EXACT = {"route": _exact_route, "route_backward": _exact_route_backward, "combine_backward": _exact_combine_backward,
          "gemm_deq": _exact_gemm_deq}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
