"""Which rows a receive buffer takes (CPU: the refusals come before any call of the library's)."""

import pytest
import torch

import combine_moe_layout_03_amd as M

BS, HIDDEN, TOPK = 4, 384, 2
IDX = torch.zeros((BS, TOPK), dtype=torch.int32)


def calls(recv):
    """Every method that fills the receive buffer, as a function of the rows."""
    quant = recv is torch.int8
    x_dtype = torch.bfloat16 if quant else recv
    one = M.EpBuffers(BS, HIDDEN, TOPK, 2, 2, x_dtype=x_dtype, quant_int8=quant, device="cpu")
    many = M.EpMultiBuffers([BS, BS], HIDDEN, TOPK, 2, 2, x_dtype=x_dtype, quant_int8=quant, device="cpu")
    return [lambda x: one.dispatch(x, IDX), lambda x: one.layout_notify_dispatch(x, IDX),
            lambda x: one.run(x, IDX, torch.zeros(BS, TOPK), fused=True), lambda x: many.dispatch(1, x, IDX)]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("x", [
    torch.zeros((BS, HIDDEN), dtype=torch.uint8),        # codes without their scales: also a whole number of lines
    torch.zeros((BS, 2 * 512), dtype=torch.uint8), torch.zeros((BS, HIDDEN), dtype=torch.bfloat16),
    torch.zeros((BS, HIDDEN)), torch.zeros(BS * 512, dtype=torch.uint8),
], ids=["codes", "wider", "bf16", "fp32", "flat"])
def test_e4m3_buffer_takes_its_own_rows_only(x, which):
    assert M.moe_recv_row_bytes(HIDDEN, M.MOE_E4M3_BLOCKSCALE) == 512
    with pytest.raises(ValueError, match=r"takes e4m3 rows, uint8 \[bs, 512\]"):
        calls(torch.float8_e4m3fn)[which](x)


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("recv", [torch.bfloat16, torch.float16, torch.int8])
def test_other_buffers_take_no_bytes(recv, which):
    with pytest.raises(ValueError, match="not one of e4m3 rows"):
        calls(recv)[which](torch.zeros((BS, 512), dtype=torch.uint8))


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("recv,x", [(torch.float8_e4m3fn, torch.zeros((BS, 512), dtype=torch.uint8)),
                                    (torch.bfloat16, torch.zeros((BS, HIDDEN), dtype=torch.bfloat16))])
def test_right_rows_reach_the_call(recv, x, which):
    with pytest.raises(ValueError, match="must be a device tensor"):
        calls(recv)[which](x)


def test_no_row_is_that_wide():
    rows = torch.zeros((1, 17024), dtype=torch.uint8)
    with pytest.raises(ValueError, match="no e4m3 row has 17024 bytes"):
        M.moe_dispatch(rows, IDX[:1], IDX[:1], IDX, IDX, 1, 1, False, rows)
