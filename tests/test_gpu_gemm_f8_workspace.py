"""The gated 8-bit float product asks for its workspace only where it passes activations through it."""

import numpy as np
import pytest
import torch

import block_rows_ref as B
import combine_moe_layout_03_amd as M
from gpu_util import log
from test_gpu_gemm_f8 import check_gated_rows, inputs, on_device

pytestmark = pytest.mark.gpu


def call(rows, k, n, counts, workspace, seed=0):
    a, ts, w, ws = inputs(np.random.default_rng(seed), rows, k, n, len(counts), 2)
    ta, rb, scale, stride, tw, tws, tc = on_device(a, ts, w, ws, counts)
    out = torch.full((rows * B.row_bytes(n),), 0xA5, dtype=torch.uint8, device="cuda")
    M.moe_grouped_gemm_swiglu_quant_f8(ta, rb, rows, k, tc, tw, tws, scale, out, workspace, token_scale_stride=stride)
    torch.cuda.synchronize()
    return out, (a, ts, w, ws, counts)


@pytest.mark.parametrize("rows,groups,n", [(1600, 2, 2048), (4096, 31, 1024), (129, 1, 12288)])
def test_whole_blocks_need_no_workspace(rows, groups, n):
    """Calls of up to 4096 rows whose workgroups hold whole blocks of 128 columns."""
    assert rows > 128 * groups and (rows // 128 + (groups + 1) // 2) * ((n + 127) // 128) >= 192
    assert M.moe_gemm_swiglu_quant_f8_workspace_bytes(rows, n) > 0
    counts = [rows - 5 * (groups - 1)] + [5] * (groups - 1)
    log(f"gemm_swiglu_f8 without a workspace {rows} {groups} {n}")
    out, case = call(rows, 128, n, counts, None)
    check_gated_rows(out, *case)


@pytest.mark.parametrize("rows,groups,n", [(128, 1, 16384), (1600, 2, 1024), (24, 16, 256)])
def test_activations_through_a_workspace_are_refused_without(rows, groups, n):
    counts = [rows] + [0] * (groups - 1)
    for workspace, status in ((None, 1), (torch.zeros(4 * rows * n - 4, dtype=torch.uint8, device="cuda"), 5)):
        with pytest.raises(M.MoeEpError) as e:
            call(rows, 16, n, counts, workspace)
        assert e.value.status == status
