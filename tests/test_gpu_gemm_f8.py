"""The block-scaled 8-bit float expert products against 64 bits, their errors
bounded by the roundings of binary32 sums."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log
from instance_cases_f8 import GATED, PLAIN, WIDE

pytestmark = pytest.mark.gpu


def codes(rng, shape, small=False):
    """e4m3 code values: normal, or whole numbers of few bits, whose products sum exactly."""
    v = rng.integers(-3, 4, shape) if small else rng.normal(size=shape) * 120
    return B.e4m3(np.clip(v, -448, 448))


def as_bytes(v):
    return torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8)


def inputs(rng, rows, k, n, groups, halves, exact=False):
    kb, nb = B.blocks(k), B.blocks(n)
    a, w = codes(rng, (rows, k), exact), codes(rng, (groups, halves * n, k), exact)
    if exact:
        ts, ws = np.ones((rows, kb)), np.ones((groups, halves * nb, kb))
    else:
        ts = (rng.random((rows, kb)) + 0.2).astype(np.float32) / 100
        ws = (rng.random((groups, halves * nb, kb)) + 0.2).astype(np.float32) / 100 / np.float32(np.sqrt(k))
    return a, ts.astype(np.float32).astype(np.float64), w, ws.astype(np.float32).astype(np.float64)


def on_device(a, ts, w, ws, counts, packed=True):
    rows, k = a.shape
    tw = as_bytes(w).cuda().view(torch.float8_e4m3fn)
    tws = torch.from_numpy(ws).float().cuda()
    tc = torch.from_numpy(np.asarray(counts, np.int32)).cuda()
    if not packed:
        return as_bytes(a).cuda(), k, torch.from_numpy(ts).float().cuda(), None, tw, tws, tc
    rb, at = B.row_bytes(k), B.scale_at(k)
    buf = torch.full((rows, rb), 0x7F, dtype=torch.uint8)  # padding of NaN codes: never part of a product
    buf[:, :k] = as_bytes(a)
    buf[:, at:at + 4 * ts.shape[1]] = torch.from_numpy(ts).float().view(torch.uint8)
    buf = buf.view(-1).cuda()
    scale, stride = M.block_scales_of(buf, k)
    return buf, rb, scale, stride, tw, tws, tc


def run_plain(a, ts, w, ws, counts, kind, packed=True, out=None):
    rows, k = a.shape
    ta, rb, scale, stride, tw, tws, tc = on_device(a, ts, w, ws, counts, packed)
    if out is None:
        out = torch.full((rows, w.shape[1]), -3.0, dtype=B.TYPES[kind], device="cuda")
    M.moe_grouped_gemm_f8(ta, rb, rows, k, tc, tw, tws, scale, out, token_scale_stride=stride)
    torch.cuda.synchronize()
    return out.float().cpu().double().numpy()


def expected(a, ts, w, ws, own, n, kind):
    """y and its error; what is rounded to 16 bits may come from the 8-bit matrix instruction."""
    y, err = B.product(a, ts, w, ws, own, n)
    return (y, err) if kind == "fp32" else (y, err + B.cut(a, ts, w, ws, own, n))


def check_plain(rng, rows, k, n, counts, kind, packed=True, exact=False):
    log(f"gemm_f8 {rows} {k} {n} {counts[:8]} {kind} exact {exact}")
    a, ts, w, ws = inputs(rng, rows, k, n, len(counts), 1, exact)
    got = run_plain(a, ts, w, ws, counts, kind, packed)
    own = B.owners(counts, rows)
    want, err = expected(a, ts, w, ws, own, n, kind)
    at = own >= 0
    if exact:  # sums of whole numbers below 2^24
        assert np.array_equal(got[at], torch.from_numpy(want[at]).to(B.TYPES[kind]).double().numpy())
    assert B.near(got[at], want[at], kind, err[at])
    assert (got[~at] == -3.0).all(), "a row of no expert was written"


def workspace(rows, n):
    size = M.moe_gemm_swiglu_quant_f8_workspace_bytes(rows, n)
    return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None


def run_gated(a, ts, w, ws, counts, packed=True):
    rows, k = a.shape
    n = w.shape[1] // 2
    ta, rb, scale, stride, tw, tws, tc = on_device(a, ts, w, ws, counts, packed)
    out = torch.full((rows * B.row_bytes(n),), 0xA5, dtype=torch.uint8, device="cuda")
    M.moe_grouped_gemm_swiglu_quant_f8(ta, rb, rows, k, tc, tw, tws, scale, out, workspace(rows, n),
                                       token_scale_stride=stride)
    torch.cuda.synchronize()
    return out


def check_gated_rows(out, a, ts, w, ws, counts):
    rows, n = a.shape[0], w.shape[1] // 2
    own = B.owners(counts, rows)
    at = own >= 0
    y, err = B.product(a, ts, w, ws, own, n)
    act, err = B.gated(y, err, n)
    got, scales = B.unpack(out, rows, n)
    B.check_rows(got[at], scales[at], act[at], err[at])
    assert (B.padding(out, rows, n) == 0xA5).all()
    raw = out.view(rows, -1).cpu().numpy()
    assert (raw[~at] == 0xA5).all(), "a row of no expert was written"


def check_gated(rng, rows, k, n, counts, packed=True):
    log(f"gemm_swiglu_f8 {rows} {k} {n} {counts[:8]}")
    a, ts, w, ws = inputs(rng, rows, k, n, len(counts), 2)
    ws *= 3  # gates on both sides of 0, some past where e^-g matters
    ws = ws.astype(np.float32).astype(np.float64)
    check_gated_rows(run_gated(a, ts, w, ws, counts, packed), a, ts, w, ws, counts)


# rows, k, n, counts: single rows, tails of k and n, experts without rows, rows of no expert, counts past the rows,
# negative counts, and rows per expert from one to many hundreds
CASES = [
    (1, 16, 16, [1]), (1, 512, 1024, [1]), (3, 16, 16, [0, 1, 0, 2]), (8, 2048, 256, [1] * 8), (24, 320, 528, [5, 0, 19]),
    (17, 48, 48, [17]), (16, 64, 64, [16]), (31, 80, 16, [15, 16]), (64, 1040, 112, [40, -3, 10]),
    (100, 128, 304, [20, 90, 50]), (130, 272, 128, [1, 129]), (257, 144, 144, [257]), (300, 256, 512, [300]),
    (700, 1024, 768, [100, 0, 350, 240]), (650, 336, 528, [300, -2, 340]), (1500, 64, 272, [700, 800]),
    (40, 160, 96, [2 ** 31 - 1, 2 ** 31 - 1]), (70, 96, 48, [0] * 130 + [1] * 70), (200, 4096, 64, [200]),
    (90, 2064, 16, [30, 30, 30]), (2, 65536, 16, [1, 1]), (520, 128, 256, [4] * 130),
]
IDS = dict(ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}-{len(c[3])}")


@pytest.mark.parametrize("case", CASES, **IDS)
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_gemm_f8(case, kind):
    rows, k, n, counts = case
    check_plain(np.random.default_rng(rows + k + n), rows, k, n - {"bf16": 0, "fp16": 3, "fp32": 15}[kind], counts, kind)


@pytest.mark.parametrize("case", CASES, **IDS)
def test_gemm_swiglu_f8(case):
    rows, k, n, counts = case
    check_gated(np.random.default_rng(rows + k + n), rows, k, n, counts)


@pytest.mark.parametrize("case", [c for c in CASES if c[1] < 60000], **IDS)
def test_gemm_f8_exact_sums(case):
    rows, k, n, counts = case
    check_plain(np.random.default_rng(k), rows, k, n, counts, "fp32", exact=True)


@pytest.mark.parametrize("name", PLAIN)
@pytest.mark.parametrize("k", [16, 128, 208, 256, 384, 528, 640, 768, 912, 1152, 2064])
def test_gemm_f8_every_kernel(name, k):
    rows, n, counts = PLAIN[name]
    check_plain(np.random.default_rng(k), rows, k, n, counts, ("bf16", "fp16")[k // 16 % 2])
    check_plain(np.random.default_rng(k), rows, k, n - 5, counts, "bf16", exact=True)


@pytest.mark.parametrize("name", WIDE)
@pytest.mark.parametrize("k", [16, 128, 208, 256, 384, 528, 640, 912, 1152])
def test_gemm_f8_every_kernel_fp32(name, k):
    rows, n, counts = WIDE[name]
    check_plain(np.random.default_rng(k), rows, k, n, counts, "fp32", exact=k % 256 == 0)


@pytest.mark.parametrize("name", PLAIN)
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_gemm_f8_every_kernel_and_type(name, kind):
    rows, n, counts = PLAIN[name]
    for k in (144, 256, 2208):
        check_plain(np.random.default_rng(k), rows, k, n, counts, kind)


@pytest.mark.parametrize("name", GATED)
@pytest.mark.parametrize("k", [16, 128, 208, 256, 384, 528, 640, 768, 912, 1152, 2064])
def test_gemm_swiglu_f8_every_kernel(name, k):
    rows, n, counts = GATED[name]
    check_gated(np.random.default_rng(k), rows, k, n, counts)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "gated"])
@pytest.mark.parametrize("rows,k,n,counts", [(100, 4096, 1280, [20, 9, 14, 16, 13, 12, 16]), (200, 4096, 1200, [90, 110]), (200, 8192, 1200, [3, 190])])
def test_gemm_f8_turned_k(rows, k, n, counts, kind):
    """A k of whole 4096s, which the experts walk from places of their own."""
    if kind == "gated":
        check_gated(np.random.default_rng(k), rows, k, n * 3 // 64 * 16, counts)
    else:
        check_plain(np.random.default_rng(k), rows, k, n - 5, counts, kind)


@pytest.mark.parametrize("rows,k,n,counts", [(20, 208, 96, [9, 11]), (300, 400, 256, [150, 150]), (900, 528, 304, [900])])
def test_gemm_f8_dense_rows_and_scales(rows, k, n, counts):
    check_plain(np.random.default_rng(n), rows, k, n, counts, "bf16", packed=False)
    check_gated(np.random.default_rng(n), rows, k, n, counts, packed=False)


def test_gemm_f8_scales_of_many_sizes():
    """Blocks whose scales differ by 2^40 and a block scaled to nothing: each block counts with its own."""
    rng = np.random.default_rng(1)
    for rows, counts in ((40, [25, 15]), (700, [400, 300])):
        a, ts, w, ws = inputs(rng, rows, 640, 160, 2, 1)
        ts *= 2.0 ** rng.integers(-20, 21, ts.shape)
        ws *= 2.0 ** rng.integers(-20, 21, ws.shape)
        ts[3], ws[1, 0, 2] = 0, 0
        log(f"gemm_f8 scales of many sizes {rows}")
        got = run_plain(a, ts, w, ws, counts, "fp32")
        want, err = B.product(a, ts, w, ws, B.owners(counts, rows), 160)
        assert B.near(got, want, "fp32", err) and (got[3] == 0).all()


def test_gemm_f8_nan_stays_in_its_row_and_column():
    """A NaN code in a row, and in a column's weights, and codes behind k that are NaN."""
    rng = np.random.default_rng(2)
    for rows, k, counts in ((40, 208, [25, 15]), (700, 336, [400, 300])):
        a, ts, w, ws = inputs(rng, rows, k, 160, 2, 1)
        ta, rb, scale, stride, tw, tws, tc = on_device(a, ts, w, ws, counts)
        ta.view(rows, rb)[7, 100] = 0x7F
        tw.view(torch.uint8)[1, 33, 5] = 0xFF
        out = torch.zeros((rows, 160), dtype=torch.float32, device="cuda")
        log(f"gemm_f8 NaN {rows}")
        M.moe_grouped_gemm_f8(ta, rb, rows, k, tc, tw, tws, scale, out, token_scale_stride=stride)
        torch.cuda.synchronize()
        own = B.owners(counts, rows)
        bad = np.zeros((rows, 160), bool)
        bad[7] = True
        bad[own == 1, 33] = True
        got = out.cpu().double().numpy()
        assert np.array_equal(np.isnan(got), bad)
        want, err = B.product(a, ts, w, ws, own, 160)
        assert B.near(got[~bad], want[~bad], "fp32", err[~bad])


def test_gemm_f8_unaligned_output():
    """An output that starts at an odd element, with rows of an odd length."""
    rng = np.random.default_rng(3)
    for rows, counts in ((60, [30, 25]), (700, [400, 290])):
        a, ts, w, ws = inputs(rng, rows, 128, 133, 2, 1)
        buf = torch.full((rows * 133 + 1,), -3.0, dtype=torch.bfloat16, device="cuda")
        log(f"gemm_f8 unaligned output {rows}")
        got = run_plain(a, ts, w, ws, counts, "bf16", out=buf[1:].view(rows, 133))
        own = B.owners(counts, rows)
        want, err = expected(a, ts, w, ws, own, 133, "bf16")
        assert B.near(got[own >= 0], want[own >= 0], "bf16", err[own >= 0])
        assert (got[own < 0] == -3.0).all() and float(buf[0]) == -3.0


def test_gemm_swiglu_f8_zero_blocks_and_large_gates():
    """Rows of zeros, whose blocks get the least scale, and gates past where e^-g overflows."""
    rng = np.random.default_rng(4)
    for rows, counts in ((40, [25, 15]), (700, [400, 300])):
        a, ts, w, ws = inputs(rng, rows, 256, 272, 2, 2)
        a[5] = 0
        ts[6] *= 1000  # gates of some hundreds
        log(f"gemm_swiglu_f8 zeros and large gates {rows}")
        out = run_gated(a, ts, w, ws, counts)
        check_gated_rows(out, a, ts, w, ws, counts)
        got, scales = B.unpack(out, rows, 272)
        assert (got[5] == 0).all() and (np.abs(scales[5] * 448 / 2.0 ** -100 - 1) <= 2 * B.U).all()


def test_gemm_f8_graph_replays_and_repeats():
    """Captured once, replayed on new rows and counts with eager calls between; the same inputs give the same bits."""
    rng = np.random.default_rng(8)
    for rows, splits in ((60, ([20, 20, 20], [0, 0, 60], [3, 50, 2])), (900, ([500, 200, 200], [0, 0, 900], [3, 850, 2]))):
        k, n = 192, 96
        a, ts, w, ws = inputs(rng, rows, k, 2 * n, 3, 1)
        _, _, w2, ws2 = inputs(rng, rows, k, n, 3, 2)
        ta, rb, scale, stride, tw, tws, tc = on_device(a, ts, w, ws, splits[0])
        tw2, tws2 = as_bytes(w2).cuda().view(torch.float8_e4m3fn), torch.from_numpy(ws2).float().cuda()
        out = torch.zeros((rows, 2 * n), dtype=torch.bfloat16, device="cuda")
        q = torch.zeros(rows * B.row_bytes(n), dtype=torch.uint8, device="cuda")
        wsp = workspace(rows, n)

        def step():
            M.moe_grouped_gemm_f8(ta, rb, rows, k, tc, tw, tws, scale, out, token_scale_stride=stride)
            M.moe_grouped_gemm_swiglu_quant_f8(ta, rb, rows, k, tc, tw2, tws2, scale, q, wsp, token_scale_stride=stride)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for r, counts in enumerate(splits):
            b = codes(rng, (rows, k))
            ta.view(rows, rb)[:, :k] = as_bytes(b).cuda()
            tc.copy_(torch.from_numpy(np.asarray(counts, np.int32)))
            out.fill_(-3.0)
            q.fill_(0xA5)
            torch.cuda.synchronize()
            log(f"gemm_f8 graph replay {rows} {r}")
            graph.replay()
            torch.cuda.synchronize()
            own = B.owners(counts, rows)
            want, err = expected(b, ts, w, ws, own, 2 * n, "bf16")
            got = out.double().cpu().numpy()
            assert B.near(got[own >= 0], want[own >= 0], "bf16", err[own >= 0]) and (got[own < 0] == -3.0).all()
            check_gated_rows(q, b, ts, w2, ws2, counts)
            first = out.clone(), q.clone()
            step()
            torch.cuda.synchronize()
            assert torch.equal(first[0], out) and torch.equal(first[1], q)


def test_gemm_f8_offsets_past_32_bits():
    """Weights, rows and outputs whose byte offsets pass 2^31 and 2^32."""
    rows, k, n, groups = 70000, 64, 32768, 2100
    log("gemm_f8 far offsets")
    gen = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randint(0, 120, (groups, n, k), dtype=torch.uint8, device="cuda", generator=gen)  # 4.4 GB, no NaN
    a = torch.randint(0, 120, (rows, k), dtype=torch.uint8, device="cuda", generator=gen)
    ws = torch.rand((groups, n // 128, 1), device="cuda", generator=gen) * 1e-4
    ts = torch.rand((rows, 1), device="cuda", generator=gen)
    counts = torch.zeros(groups, dtype=torch.int32, device="cuda")
    counts[3], counts[2098], counts[2099] = 69000, 1, 999
    out = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    M.moe_grouped_gemm_f8(a, k, rows, k, counts, w, ws, ts, out)
    torch.cuda.synchronize()
    values = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    for r, g in ((0, 3), (33000, 3), (68999, 3), (69000, 2098), (69001, 2099), (69999, 2099)):
        y = (values[w[g].long()] @ values[a[r].long()]) * ws[g].double().repeat_interleave(128, 0)[:, 0] * ts[r].double()
        # every term is positive: 140 roundings of binary32, half a step of bf16, and seven cuts of 2^-13
        assert (((out[r].double() - y).abs() / y) <= 140 * B.U + 2.0 ** -8 + 7 * 2.0 ** -13).all(), r


def test_gemm_swiglu_f8_offsets_past_32_bits():
    rows, k, n, groups = 70000, 32, 32768, 2100
    log("gemm_swiglu_f8 far offsets")
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randint(0, 100, (groups, 2 * n, k), dtype=torch.uint8, device="cuda", generator=gen)  # 4.4 GB
    a = torch.randint(0, 100, (rows, k), dtype=torch.uint8, device="cuda", generator=gen)
    ws = torch.rand((groups, 2 * n // 128, 1), device="cuda", generator=gen) * 1e-3
    ts = torch.rand((rows, 1), device="cuda", generator=gen)
    counts = torch.zeros(groups, dtype=torch.int32, device="cuda")
    counts[3], counts[2098], counts[2099] = 69000, 1, 999
    out = torch.zeros(rows * B.row_bytes(n), dtype=torch.uint8, device="cuda")
    M.moe_grouped_gemm_swiglu_quant_f8(a, k, rows, k, counts, w, ws, ts, out, workspace(rows, n))
    torch.cuda.synchronize()
    values = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    m = out.view(rows, -1)
    for r, g in ((0, 3), (33000, 3), (68999, 3), (69000, 2098), (69001, 2099), (69999, 2099)):
        y = (values[w[g].long()] @ values[a[r].long()]) * ws[g].double().repeat_interleave(128, 0)[:, 0] * ts[r].double()
        gate, up = y[:n], y[n:]
        act = gate * torch.sigmoid(gate) * up
        got, scales = B.unpack(m[r].contiguous(), 1, n)
        # every term is positive: 42 roundings in a factor, whose slopes are at most 1.3 relative
        B.check_rows(got, scales, act.cpu().numpy()[None], 120 * B.U * act.cpu().numpy()[None])
