"""Host-side refusals of the norm, its gradient and the 8-bit float products (no
GPU: each call returns before any HIP call), and the binding's own checks."""

import ctypes

import pytest
import torch

import combine_moe_layout_03_amd as M

P = 0x100000  # a non-NULL, aligned stand-in pointer, never dereferenced


@pytest.mark.parametrize("hidden,expect", [(16, 128), (96, 128), (112, 256), (128, 256), (1040, 1152), (2048, 2176),
                                           (7168, 7424), (16384, 16896)])
def test_row_bytes(hidden, expect):
    assert M.moe_recv_row_bytes(hidden, M.MOE_E4M3_BLOCKSCALE) == expect


def norm(**kw):
    a = dict(x=P, r=P, t=0, w=P, eps=1e-6, bs=16, h=1024, s=P, o=P, ot=0, rows=P, rb=16 * 1152, rs=P)
    a.update(kw)
    return M._lib.moe_rms_norm(a["x"], a["r"], a["t"], a["w"], a["eps"], a["bs"], a["h"], a["s"], a["o"], a["ot"],
                               a["rows"], a["rb"], a["rs"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(bs=-1), 2), (dict(h=0), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(h=1020), 7), (dict(h=16392), 7), (dict(h=1032), 7), (dict(t=3), 4), (dict(t=4), 4), (dict(ot=3), 4),
    (dict(x=None), 1), (dict(w=None), 1), (dict(o=None, rows=None), 1),
    (dict(x=P + 8), 3), (dict(r=P + 8), 3), (dict(w=P + 2), 3), (dict(s=P + 8), 3), (dict(o=P + 8), 3),
    (dict(rows=P + 8), 3), (dict(rs=P + 2), 3), (dict(rb=16 * 1152 - 1), 6),
])
def test_norm_rejects(bad, status):
    assert norm(**bad) == status


def test_norm_empty_batch():
    assert norm(bs=0, x=None, w=None, o=None, rows=None) == 0


def backward(**kw):
    a = dict(g=P, gt=0, gs=P, s=P, t=0, w=P, rs=P, m=P, bs=16, h=1024, d=P, dw=P, ws=P, wb=2 * 1024 * 4)
    a.update(kw)
    return M._lib.moe_rms_norm_backward(a["g"], a["gt"], a["gs"], a["s"], a["t"], a["w"], a["rs"], a["m"], a["bs"],
                                        a["h"], a["d"], a["dw"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(bs=-1), 2), (dict(h=0), 2), (dict(h=1020), 7), (dict(h=16392), 7), (dict(t=3), 4), (dict(gt=4), 4),
    (dict(g=None), 1), (dict(s=None), 1), (dict(w=None), 1), (dict(rs=None), 1), (dict(d=None), 1), (dict(ws=None), 1),
    (dict(g=P + 8), 3), (dict(gs=P + 8), 3), (dict(s=P + 8), 3), (dict(w=P + 2), 3), (dict(rs=P + 2), 3),
    (dict(d=P + 8), 3), (dict(dw=P + 2), 3), (dict(ws=P + 8), 3), (dict(wb=2 * 1024 * 4 - 1), 5),
])
def test_norm_backward_rejects(bad, status):
    assert backward(**bad) == status


def test_norm_backward_workspace():
    assert backward(bs=0, g=None, s=None, w=None, rs=None, d=None, dw=None, ws=None, wb=0) == 0
    assert M.moe_rms_norm_backward_workspace_bytes(0, 64) == 0
    assert M.moe_rms_norm_backward_workspace_bytes(5, 64) == 64 * 4
    assert M.moe_rms_norm_backward_workspace_bytes(2 ** 31 - 1, 16384) == 256 * 16384 * 4
    size = ctypes.c_size_t()
    assert M._lib.moe_rms_norm_backward_workspace_bytes(-1, 64, ctypes.byref(size)) == 2
    assert M._lib.moe_rms_norm_backward_workspace_bytes(1, 63, ctypes.byref(size)) == 7
    assert M._lib.moe_rms_norm_backward_workspace_bytes(1, 64, None) == 1


GEMM = dict(a=P, ab=2176, rows=64, k=2048, gc=P, g=4, w=P, n=1008, ws=P, ts=P, st=2176, out=P, wsp=P, wb=1 << 40)


def gemm(**kw):
    a = dict(GEMM, ot=0, ob=64 * 1008 * 2)
    a.update(kw)
    return M._lib.moe_grouped_gemm_f8(a["a"], a["ab"], a["rows"], a["k"], a["gc"], a["g"], a["w"], a["n"], a["ws"],
                                      a["ts"], a["st"], a["out"], a["ot"], a["ob"], None)


def gated(**kw):
    a = dict(GEMM, ob=64 * 1152)
    a.update(kw)
    return M._lib.moe_grouped_gemm_swiglu_quant_f8(a["a"], a["ab"], a["rows"], a["k"], a["gc"], a["g"], a["w"], a["n"],
                                                   a["ws"], a["ts"], a["st"], a["out"], a["ob"], a["wsp"], a["wb"], None)


BOTH = [
    (dict(rows=-1), 2), (dict(k=0), 2), (dict(n=0), 2), (dict(g=0), 2), (dict(ab=2032), 2), (dict(st=60), 2),
    (dict(st=0), 2), (dict(st=-64), 2), (dict(st=66), 2), (dict(k=2040), 7), (dict(k=65552, ab=65552), 7),
    (dict(g=65537), 7), (dict(ab=2 ** 23 + 16), 7), (dict(ab=2184), 3), (dict(a=None), 1), (dict(gc=None), 1), (dict(w=None), 1),
    (dict(ws=None), 1), (dict(ts=None), 1), (dict(out=None), 1), (dict(a=P + 8), 3), (dict(w=P + 8), 3),
    (dict(gc=P + 2), 3), (dict(ws=P + 2), 3), (dict(ts=P + 2), 3),
]


@pytest.mark.parametrize("bad,status", BOTH + [
    (dict(n=65537), 7), (dict(ot=3), 4), (dict(ot=4), 4), (dict(out=P + 1), 3), (dict(out=P + 2, ot=2, ob=64 * 4032), 3),
    (dict(ob=64 * 1008 * 2 - 1), 6), (dict(ot=2), 6),
    (dict(rows=2 ** 31 - 1, n=65536, ob=2 ** 48), 7),  # more workgroups than one launch takes
])
def test_gemm_f8_rejects(bad, status):
    assert gemm(**bad) == status


@pytest.mark.parametrize("bad,status", BOTH + [
    (dict(n=1000), 7), (dict(n=32784), 7), (dict(out=P + 8), 3), (dict(wsp=P + 8), 3), (dict(ob=64 * 1152 - 1), 6),
    (dict(rows=2 ** 31 - 1, n=32768, ob=2 ** 48), 7),
])
def test_gemm_swiglu_f8_rejects(bad, status):
    assert gated(**bad) == status


def test_no_rows():
    assert gemm(rows=0, a=None, out=None, ob=0) == 0
    assert gated(rows=0, a=None, out=None, ob=0, wsp=None, wb=0) == 0


def test_gated_workspace():
    size = M.moe_gemm_swiglu_quant_f8_workspace_bytes
    assert all(size(r, n) <= 4 * min(r, 4096) * n for r in (0, 1, 17, 5000, 2 ** 31 - 1) for n in (16, 2048, 32768))
    need = size(64, 1008)
    if need:
        assert gated(wb=need - 1) == 5 and gated(wsp=None) == 1
    out = ctypes.c_size_t()
    assert M._lib.moe_gemm_swiglu_quant_f8_workspace_bytes(-1, 16, ctypes.byref(out)) == 2
    assert M._lib.moe_gemm_swiglu_quant_f8_workspace_bytes(1, 0, ctypes.byref(out)) == 2
    assert M._lib.moe_gemm_swiglu_quant_f8_workspace_bytes(1, 16, None) == 1


def dispatch(**kw):
    need = 16 * 8 * 1152
    a = dict(x=P, t=4, bs=16, h=1024, k=8, q=0, recv=P, rb=need)
    a.update(kw)
    return M._lib.moe_dispatch(a["x"], a["t"], a["bs"], a["h"], a["k"], P, P, P, P, 4, 4, a["q"], a["recv"], a["rb"],
                               None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=1), 4), (dict(h=0), 2), (dict(h=1032), 7), (dict(h=16400), 7), (dict(rb=16 * 8 * 1152 - 1), 6),
    (dict(x=None), 1), (dict(t=5), 4),
])
def test_dispatch_of_e4m3_rows_rejects(bad, status):
    assert dispatch(**bad) == status


def test_fused_supported_by_the_rows_bytes():
    assert M.moe_fused_supported(16, 7168, 8, 16, 16, torch.float8_e4m3fn, False)
    assert M.moe_fused_supported(16, 15872, 8, 16, 16, torch.float8_e4m3fn, False)  # rows of 16384 bytes
    assert not M.moe_fused_supported(16, 15888, 8, 16, 16, torch.float8_e4m3fn, False)
    with pytest.raises(M.MoeEpError):
        M.moe_fused_supported(16, 7168, 8, 16, 16, torch.float8_e4m3fn, True)


def test_binding_checks():
    """The binding refuses host tensors and wrong shapes before the call."""
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        M.moe_rms_norm(x, w, 1e-6, out=x)
    with pytest.raises(ValueError, match="grad_out must be a device tensor"):
        M.moe_rms_norm_backward(x, x, w, w, x)
    rows, codes = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(1, 4, 16, dtype=torch.uint8)
    count, scale = torch.zeros(1, dtype=torch.int32), torch.zeros(4, 1)
    with pytest.raises(ValueError, match=r"w must be e4m3 \[groups, n, k\]"):
        M.moe_grouped_gemm_f8(rows, 16, 4, 16, count, torch.zeros(1, 4, 32, dtype=torch.uint8), scale, scale, x)
    with pytest.raises(ValueError, match=r"w must be e4m3 \[groups, 2n, k\]"):
        M.moe_grouped_gemm_swiglu_quant_f8(rows, 16, 4, 16, count, codes[:, :3], scale, scale, rows)
    with pytest.raises(ValueError, match="weight_scale must hold"):
        M.moe_grouped_gemm_f8(rows, 16, 4, 16, count, codes, scale, scale, x)
    with pytest.raises(ValueError, match="group_count must hold"):
        M.moe_grouped_gemm_f8(rows, 16, 4, 16, torch.zeros(2, dtype=torch.int32), codes, scale[:1], scale, x)
    with pytest.raises(ValueError, match="a is smaller"):
        M.moe_grouped_gemm_f8(rows, 32, 4, 16, count, codes, scale[:1], scale, x)
    with pytest.raises(ValueError, match="token_scale must be contiguous"):
        M.moe_grouped_gemm_f8(rows, 16, 4, 16, count, codes, scale[:1], scale.double(), x)
    with pytest.raises(ValueError, match="token_scale must be a device tensor"):
        M.moe_grouped_gemm_f8(rows, 16, 4, 16, count, codes, scale[:1], scale, x)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="as they are"):
        M.moe_dispatch(torch.zeros(4, 256, dtype=torch.uint8), idx, idx, idx, idx, 1, 1, True, rows)
    with pytest.raises(ValueError, match="whole lines"):
        M.moe_dispatch(torch.zeros(4, 200, dtype=torch.uint8), idx, idx, idx, idx, 1, 1, False, rows)
