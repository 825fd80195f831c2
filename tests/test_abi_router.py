"""Host-side refusals of the router, the gradients and the scaled expert
product (no GPU: each call returns before any HIP call), and the binding's
own checks."""

import pytest
import torch

import combine_moe_layout_03_amd as M

P = 0x100000  # a non-NULL, aligned stand-in pointer, never dereferenced


def route(**kw):
    a = dict(x=P, t=2, st=256, bs=16, e=256, k=8, score=1, bias=P, g=8, keep=4, top=2, re=1, mask=None, idx=P, w=P)
    a.update(kw)
    return M._lib.moe_route(a["x"], a["t"], a["st"], a["bs"], a["e"], a["k"], a["score"], a["bias"], a["g"], a["keep"],
                            a["top"], a["re"], 1.0, a["mask"], a["idx"], a["w"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(bs=-1), 2), (dict(e=0), 2), (dict(k=0), 2), (dict(st=255), 2), (dict(g=0), 2), (dict(keep=0), 2),
    (dict(keep=9), 2), (dict(g=7), 2), (dict(top=0), 2), (dict(top=3), 2), (dict(k=32, keep=1, g=16), 2),
    (dict(k=257, g=1, keep=1, st=257), 2),
    (dict(e=2049, st=2049, g=1, keep=1), 7), (dict(e=2048, st=2048, g=1, keep=1, k=33), 7),
    (dict(e=260, st=260, g=65, keep=65), 7), (dict(bs=2 ** 28), 7),
    (dict(t=3), 4), (dict(score=2), 4), (dict(score=-1), 4), (dict(re=2), 4),
    (dict(x=None), 1), (dict(idx=None), 1), (dict(w=None), 1),
    (dict(x=P + 2), 3), (dict(x=P + 1, t=0), 3), (dict(bias=P + 2), 3), (dict(idx=P + 1), 3), (dict(w=P + 2), 3),
])
def test_route_rejects(bad, status):
    assert route(**bad) == status


def test_route_empty_batch():
    assert route(bs=0, x=None, idx=None, w=None) == 0


def backward(**kw):
    a = dict(g=P, x=P, t=2, st=256, idx=P, bs=16, e=256, k=8, score=0, re=0, d=P, ds=256)
    a.update(kw)
    return M._lib.moe_route_backward(a["g"], a["x"], a["t"], a["st"], a["idx"], a["bs"], a["e"], a["k"], a["score"],
                                     a["re"], 1.0, a["d"], a["ds"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(bs=-1), 2), (dict(e=0), 2), (dict(k=0), 2), (dict(k=257), 2), (dict(st=255), 2), (dict(ds=255), 2),
    (dict(e=4096, st=4096, ds=4096), 7), (dict(k=33), 7), (dict(t=3), 4), (dict(score=5), 4), (dict(re=-1), 4),
    (dict(g=None), 1), (dict(x=None), 1), (dict(idx=None), 1), (dict(d=None), 1),
    (dict(g=P + 2), 3), (dict(x=P + 2), 3), (dict(idx=P + 2), 3), (dict(d=P + 2), 3), (dict(d=P + 1, t=1), 3),
])
def test_route_backward_rejects(bad, status):
    assert backward(**bad) == status


def test_route_backward_empty_batch():
    assert backward(bs=0, g=None, x=None, idx=None, d=None) == 0


def combine_backward(**kw):
    need = 16 * 8 * 2 * 1024
    a = dict(go=P, gt=0, x=P, rt=0, xb=need, bs=16, h=1024, k=8, idx=P, w=P, slot=P, put=P, base=P, epr=4, r=4, ns=3,
             src=1, gr=P, gb=need, gw=P)
    a.update(kw)
    head = (a["go"], a["gt"], a["x"], a["rt"], a["xb"], a["bs"], a["h"], a["k"], a["idx"], a["w"], a["slot"],
            a["put"], a["base"], a["epr"], a["r"])
    many = M._lib.moe_combine_backward_src(*head, a["ns"], a["src"], a["gr"], a["gb"], a["gw"], None)
    if a["ns"] == 3 and a["src"] == 1:
        assert M._lib.moe_combine_backward(*head, a["gr"], a["gb"], a["gw"], None) == many
    return many


@pytest.mark.parametrize("bad,status", [
    (dict(rt=2), 4), (dict(rt=3), 4), (dict(gt=3), 4), (dict(bs=-1), 2), (dict(k=0), 2), (dict(k=33), 7),
    (dict(h=1020), 7), (dict(h=0), 2), (dict(h=16392), 7), (dict(epr=0), 2), (dict(epr=1024), 7),
    (dict(ns=0, src=0), 2), (dict(src=3), 2), (dict(src=-1), 2), (dict(ns=385), 7),
    (dict(xb=16 * 8 * 2 * 1024 - 1), 6), (dict(gb=16 * 8 * 2 * 1024 - 1), 6),
    (dict(go=None), 1), (dict(x=None), 1), (dict(idx=None), 1), (dict(w=None), 1), (dict(slot=None), 1),
    (dict(gr=None), 1), (dict(gw=None), 1),
    (dict(go=P + 8), 3), (dict(x=P + 8), 3), (dict(gr=P + 8), 3), (dict(w=P + 2), 3), (dict(gw=P + 2), 3),
    (dict(put=P + 2), 3),
])
def test_combine_backward_rejects(bad, status):
    assert combine_backward(**bad) == status


def test_combine_backward_empty_batch():
    assert combine_backward(bs=0, go=None, x=None, w=None, gr=None, gw=None, idx=None, xb=0, gb=0) == 0


def gemm(**kw):
    a = dict(a=P, ab=2176, rows=64, k=2048, gc=P, g=4, w=P, n=1000, ws=P, ts=P, st=2176, out=P, ot=0, ob=64 * 1000 * 2)
    a.update(kw)
    return M._lib.moe_grouped_gemm_deq_i8(a["a"], a["ab"], a["rows"], a["k"], a["gc"], a["g"], a["w"], a["n"], a["ws"],
                                          a["ts"], a["st"], a["out"], a["ot"], a["ob"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), 2), (dict(k=0), 2), (dict(n=0), 2), (dict(g=0), 2), (dict(ab=2032), 2), (dict(st=0), 2),
    (dict(st=6), 2), (dict(k=2040), 7), (dict(k=65552, ab=65552), 7), (dict(n=65537), 7), (dict(g=65537), 7),
    (dict(ot=3), 4), (dict(ab=2184), 3), (dict(a=None), 1), (dict(gc=None), 1), (dict(w=None), 1), (dict(ws=None), 1),
    (dict(ts=None), 1), (dict(out=None), 1), (dict(a=P + 8), 3), (dict(w=P + 8), 3), (dict(gc=P + 2), 3),
    (dict(ws=P + 2), 3), (dict(ts=P + 2), 3), (dict(out=P + 1), 3), (dict(out=P + 2, ot=2, ob=64 * 4000), 3),
    (dict(ob=64 * 1000 * 2 - 1), 6), (dict(ot=2), 6),
    (dict(rows=2 ** 31 - 1, n=65536, ob=2 ** 48), 7),  # more workgroups than one launch takes
])
def test_gemm_deq_rejects(bad, status):
    assert gemm(**bad) == status


def test_gemm_deq_no_rows():
    assert gemm(rows=0, a=None, out=None, ob=0) == 0


def test_binding_checks():
    """The binding refuses host tensors and wrong shapes before the call."""
    x, idx, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="logits must be a device tensor"):
        M.moe_route(x, idx, w, M.MOE_SCORE_SOFTMAX)
    with pytest.raises(ValueError, match="logits must be a device tensor"):
        M.moe_route_backward(w, x, idx, M.MOE_SCORE_SOFTMAX, x)
    with pytest.raises(ValueError, match=r"grad_out must be \[bs, hidden\]"):
        M.moe_combine_backward(x, x, M.MOE_BF16, idx[:3], w, idx, idx, idx, 2, 4, x, w)
    with pytest.raises(ValueError, match="send_token_idx holds 3 elements"):
        M.moe_combine_backward(x, x, M.MOE_BF16, idx, w, idx.view(-1)[:3], idx, idx, 2, 4, x, w)
    with pytest.raises(ValueError, match=r"put_offset must be \[E, num_src\]"):
        M.moe_combine_backward_src(x, x, M.MOE_BF16, idx, w, idx, idx.view(-1), idx, 2, 4, 0, x, w)
    bad = torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="w must be int8"):
        M.moe_grouped_gemm_deq_i8(bad, 16, 4, 16, idx, torch.zeros(1, 4, 32, dtype=torch.int8), w, w, x)
    with pytest.raises(ValueError, match="weight_scale must hold"):
        M.moe_grouped_gemm_deq_i8(bad, 16, 4, 16, idx.view(-1)[:1], torch.zeros(1, 4, 16, dtype=torch.int8), w, w, x)
