"""The scaled int8 expert product, bit for bit against its definition: exact
integer sums (64 bits), then two binary32 products and one rounding."""

import numpy as np
import pytest
import torch

import combine_moe_layout_03_amd as M
import router_ref as R
from gpu_util import align32, int8_row_bytes, log
from instance_cases_deq import TILED

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def inputs(rng, rows, k, n, groups, full=False):
    if full:  # every product at its largest: the sums reach k * 2^14
        a = np.full((rows, k), -128, np.int8)
        w = np.full((groups, n, k), -128, np.int8)
        w[:, ::2] = 127
    else:
        a = rng.integers(-128, 128, (rows, k)).astype(np.int8)
        w = rng.integers(-128, 128, (groups, n, k)).astype(np.int8)
    ws = (rng.random((groups, n)) * 0.01 + 1e-4).astype(np.float32)
    ts = (rng.random(rows) * 0.02 + 1e-4).astype(np.float32)
    return a, w, ws, ts


def owners(counts, rows):
    """Expert of each row, -1 for none."""
    got = np.full(rows, -1)
    at = 0
    for g, c in enumerate(counts):
        c = max(int(c), 0)
        got[min(at, rows):min(at + c, rows)] = g
        at += c
    return got


def expected(a, w, ws, ts, counts, kind):
    rows, n = a.shape[0], w.shape[1]
    own = owners(counts, rows)
    out = np.zeros((rows, n), np.float32)
    for g in range(w.shape[0]):
        at = np.nonzero(own == g)[0]
        if len(at):
            acc = (a[at].astype(np.float64) @ w[g].astype(np.float64).T).astype(np.int64)  # exact: below 2^53
            out[at] = acc.astype(np.float32) * ws[g] * ts[at, None]
    return R.to_type(out, kind), own


def run(a, w, ws, ts, counts, kind, packed=True, out=None):
    rows, k = a.shape
    n = w.shape[1]
    if packed:  # the receive-buffer form, its inverse scales in place
        rb = int8_row_bytes(k)
        buf = np.full((rows, rb), 0x5A, np.uint8)
        buf[:, :k] = a.view(np.uint8)
        buf[:, align32(k):align32(k) + 4] = ts.view(np.uint8).reshape(rows, 4)
        ta = torch.from_numpy(buf.reshape(-1)).cuda()
        scale, stride = M.token_scales_of(ta, k)
    else:
        rb = k
        ta = torch.from_numpy(np.ascontiguousarray(a)).cuda()
        scale, stride = torch.from_numpy(ts).cuda(), 4
    if out is None:
        out = torch.full((rows, n), -3.0, dtype=TYPES[kind], device="cuda")
    M.moe_grouped_gemm_deq_i8(ta.view(-1), rb, rows, k, torch.from_numpy(np.asarray(counts, np.int32)).cuda(),
                              torch.from_numpy(w).cuda(), torch.from_numpy(ws).cuda(), scale, out,
                              token_scale_stride=stride)
    torch.cuda.synchronize()
    return out.float().cpu().numpy()


def check(rng, rows, k, n, counts, kind, packed=True, full=False):
    a, w, ws, ts = inputs(rng, rows, k, n, len(counts), full)
    got = run(a, w, ws, ts, counts, kind, packed)
    want, own = expected(a, w, ws, ts, counts, kind)
    assert np.array_equal(got[own >= 0], want[own >= 0])
    assert (got[own < 0] == -3.0).all(), "a row of no expert was written"


# rows, k, n, counts: single rows, tails of k and n, experts without rows, rows of no expert, counts past the rows,
# negative counts, and rows per expert from one to many hundreds
CASES = [
    (1, 16, 1, [1]), (1, 512, 1024, [1]), (3, 16, 16, [0, 1, 0, 2]), (8, 2048, 256, [1] * 8), (24, 320, 520, [5, 0, 19]),
    (17, 48, 33, [17]), (16, 64, 64, [16]), (31, 80, 17, [15, 16]), (64, 1040, 100, [40, -3, 10]),
    (100, 128, 300, [20, 90, 50]), (130, 272, 129, [1, 129]), (257, 144, 130, [257]), (300, 256, 512, [300]),
    (700, 1024, 768, [100, 0, 350, 240]), (650, 336, 515, [300, -2, 340]), (1500, 64, 260, [700, 800]),
    (40, 160, 96, [2 ** 31 - 1, 2 ** 31 - 1]), (70, 96, 40, [0] * 130 + [1] * 70), (200, 4096, 64, [200]),
    (90, 2064, 1, [30, 30, 30]), (2, 65536, 8, [1, 1]), (520, 128, 256, [4] * 130),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}-{len(c[3])}")
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_gemm_deq(case, kind):
    rows, k, n, counts = case
    log(f"gemm_deq {rows} {k} {n} {counts[:8]} {kind}")
    check(np.random.default_rng(rows + k + n), rows, k, n, counts, kind)


@pytest.mark.parametrize("rows,k,n,counts", [(20, 208, 90, [9, 11]), (300, 400, 257, [150, 150]), (900, 528, 300, [900])])
def test_gemm_deq_dense_rows_and_scales(rows, k, n, counts):
    log(f"gemm_deq dense {rows} {k} {n}")
    check(np.random.default_rng(n), rows, k, n, counts, "bf16", packed=False)


@pytest.mark.parametrize("rows,k,n,counts", [(5, 65536, 16, [2, 3]), (300, 65536, 16, [300])])
def test_gemm_deq_largest_sums(rows, k, n, counts):
    log(f"gemm_deq largest sums {rows} {k} {n}")
    check(np.random.default_rng(1), rows, k, n, counts, "fp32", full=True)


def test_gemm_deq_overflow_and_subnormals():
    """fp16 overflows to infinity, and products below the normal range keep binary32's subnormals."""
    rng = np.random.default_rng(2)
    a, w, ws, ts = inputs(rng, 40, 64, 48, 2)
    ts[:20] = 1e6
    ts[20:] = 1e-38
    for kind in ("fp16", "fp32", "bf16"):
        log(f"gemm_deq extremes {kind}")
        got, (want, own) = run(a, w, ws, ts, [21, 19], kind), expected(a, w, ws, ts, [21, 19], kind)
        assert np.array_equal(got, want)


def test_gemm_deq_unaligned_output_and_streams():
    """An output that starts at an odd element, on a stream of the caller's."""
    rng = np.random.default_rng(3)
    a, w, ws, ts = inputs(rng, 300, 128, 133, 2)
    buf = torch.full((300 * 133 + 1,), -3.0, dtype=torch.bfloat16, device="cuda")
    log("gemm_deq unaligned output")
    got = run(a, w, ws, ts, [200, 90], "bf16", out=buf[1:].view(300, 133))
    want, own = expected(a, w, ws, ts, [200, 90], "bf16")
    assert np.array_equal(got[own >= 0], want[own >= 0]) and (got[own < 0] == -3.0).all() and float(buf[0]) == -3.0


def test_gemm_deq_offsets_past_32_bits():
    """Weights, rows and outputs whose byte offsets pass 2^31 and 2^32."""
    rows, k, n, groups = 70000, 64, 32768, 2100
    log("gemm_deq far offsets")
    gen = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randint(-128, 128, (groups, n, k), dtype=torch.int8, device="cuda", generator=gen)  # 4.4 GB
    a = torch.randint(-128, 128, (rows, k), dtype=torch.int8, device="cuda", generator=gen)
    ws = torch.rand((groups, n), device="cuda", generator=gen)
    ts = torch.rand((rows,), device="cuda", generator=gen)
    counts = torch.zeros(groups, dtype=torch.int32, device="cuda")
    counts[3], counts[2098], counts[2099] = 69000, 1, 999
    out = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    M.moe_grouped_gemm_deq_i8(a.view(-1), k, rows, k, counts, w, ws, ts, out)
    torch.cuda.synchronize()
    for r, g in ((0, 3), (33000, 3), (68999, 3), (69000, 2098), (69001, 2099), (69999, 2099)):
        acc = (w[g].double() @ a[r].double()).float()
        assert torch.equal(out[r], (acc * ws[g] * ts[r]).bfloat16()), r


def test_gemm_deq_graph_replays():
    """Captured once, replayed on new rows and counts with eager calls between."""
    rng = np.random.default_rng(8)
    rows, k, n, groups = 200, 192, 96, 3
    a, w, ws, ts = inputs(rng, rows, k, n, groups)
    ta = torch.from_numpy(a).cuda()
    tw, tws, tts = (torch.from_numpy(v).cuda() for v in (w, ws, ts))
    tc = torch.zeros(groups, dtype=torch.int32, device="cuda")
    out = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")

    def step():
        M.moe_grouped_gemm_deq_i8(ta.view(-1), k, rows, k, tc, tw, tws, tts, out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.zeros_like(out)
    for r, counts in enumerate(([100, 50, 50], [0, 0, 200], [3, 150, 2])):
        b = rng.integers(-128, 128, (rows, k)).astype(np.int8)
        ta.copy_(torch.from_numpy(b))
        tc.copy_(torch.from_numpy(np.asarray(counts, np.int32)))
        out.fill_(-3.0)
        torch.cuda.synchronize()
        log(f"gemm_deq graph replay {r}")
        graph.replay()
        torch.cuda.synchronize()
        want, own = expected(b, w, ws, ts, counts, "bf16")
        got = out.float().cpu().numpy()
        assert np.array_equal(got[own >= 0], want[own >= 0]) and (got[own < 0] == -3.0).all()
        M.moe_grouped_gemm_deq_i8(ta.view(-1), k, rows, k, tc, tw, tws, tts, other)
        torch.cuda.synchronize()


@pytest.mark.parametrize("tile", TILED)
@pytest.mark.parametrize("k", [16, 128, 208, 256, 384, 528, 640, 768, 912, 1024, 1152, 2064, 2560, 3600])
def test_gemm_deq_every_tile(tile, k):
    """Every tile at every number of stages that its loop's rounds can leave."""
    rows, n, counts = TILED[tile]
    kind = ("bf16", "fp16", "fp32")[k // 16 % 3]
    log(f"gemm_deq {tile} k {k} {kind}")
    check(np.random.default_rng(k), rows, k, n, counts, kind)


@pytest.mark.parametrize("tile", TILED)
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_gemm_deq_every_tile_and_type(tile, kind):
    rows, n, counts = TILED[tile]
    log(f"gemm_deq {tile} {kind}")
    for k in (144, 256, 2208):
        check(np.random.default_rng(k), rows, k, n, counts, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_gemm_deq_large_weights(kind):
    """Weights past what the caches keep (the results are then stored non-temporally), odd rows at odd addresses."""
    rows, n, counts = TILED["tile64"]
    log(f"gemm_deq large weights {kind}")
    check(np.random.default_rng(9), rows, 4112, n - 1, counts, kind)


@pytest.mark.parametrize("tile", TILED)
def test_gemm_deq_turned_k(tile):
    """A k of whole 4096s, which the experts and columns walk from places of their own."""
    rows, n, counts = TILED[tile]
    log(f"gemm_deq {tile} k 4096")
    check(np.random.default_rng(10), rows, 4096, n, counts, "bf16")
