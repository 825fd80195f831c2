"""The expert products refuse more threads than one launch takes (2^32 - 1) on the host, before any HIP call (CPU only:
every call here is refused)."""

import pytest

import combine_moe_layout_03_amd as M

P = 0x100000  # a non-NULL, aligned stand-in pointer, never dereferenced
UNSUPPORTED = 7


# rows, groups, n of launches with 2^23 workgroups of 512 threads or a few more, below the 2^24 workgroups that a grid
# could have otherwise
@pytest.mark.parametrize("rows,groups,n", [(2 ** 31 - 1, 2, 1), (2 ** 31 - 1, 1, 200), (2 ** 30, 1, 257), (2 ** 30, 9, 500)])
def test_tiles_of_256_rows(rows, groups, n):
    deq = M._lib.moe_grouped_gemm_deq_i8(P, 16, rows, 16, P, groups, P, n, P, P, 4, P, M.MOE_FP32, rows * n * 4, None)
    assert deq == UNSUPPORTED
    assert M._lib.moe_grouped_gemm_i8(P, 16, rows, 16, P, groups, P, n, P, rows * n * 4, None) == UNSUPPORTED


@pytest.mark.parametrize("rows,groups,n", [(2 ** 31 - 1, 2, 4), (2 ** 30, 1, 132)])
def test_fused_product(rows, groups, n):
    out = rows * M.moe_recv_row_bytes(n, M.MOE_INT8_ROWSCALE)
    space = M.moe_gemm_swiglu_quant_workspace_bytes(rows, n)
    assert M._lib.moe_grouped_gemm_swiglu_quant_i8(P, 16, rows, 16, P, groups, P, n, P, P, 4, P, out, P, space,
                                                   None) == UNSUPPORTED


def test_streams():
    """2^24 workgroups of 256 threads (tiles of 16 rows and 32 columns, 65536 experts of a row or two each)."""
    rows = 65536
    slots = rows // 16 + 65536
    n = 32 * 8 * (-(-2 ** 24 // (slots * 8)))  # whole eighths of column tiles
    assert slots * (n // 32) >= 2 ** 24 and slots * (n // 32 - 8) < 2 ** 24
    assert M._lib.moe_grouped_gemm_deq_i8(P, 2048, rows, 2048, P, 65536, P, n, P, P, 4, P, M.MOE_BF16, rows * n * 2,
                                          None) == UNSUPPORTED
