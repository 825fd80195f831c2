"""The norm and the 8-bit float products refuse every tensor of another device than the current one, on whose stream
they run (CPU: tensors that say where they are, and a library that is not called)."""

import inspect

import pytest
import torch

import combine_moe_layout_03_amd as M

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32


class On(torch.Tensor):
    """A host tensor that says it is a device's."""
    at = 0
    is_cuda = True

    def get_device(self):
        return self.at


def tensor(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(On)


CALLS = {
    "moe_rms_norm": dict(x=((4, 16), BF16), weight=(16, F32), residual=((4, 16), BF16), sum=((4, 16), BF16),
                         out=((4, 16), BF16), rows=(4 * 128, U8), rstd=(4, F32)),
    "moe_rms_norm_backward": dict(grad_out=((4, 16), BF16), sum=((4, 16), BF16), weight=(16, F32), rstd=(4, F32),
                                  grad_x=((4, 16), BF16), grad_sum=((4, 16), BF16), grad_weight=(16, F32),
                                  workspace=(64, U8), token_mask=(4, U8)),
    "moe_grouped_gemm_f8": dict(a=(4 * 128, U8), group_count=(2, I32), w=((2, 16, 16), U8), weight_scale=((2, 1, 1), F32),
                                token_scale=(4, F32), out=((4, 16), BF16)),
    "moe_grouped_gemm_swiglu_quant_f8": dict(a=(4 * 128, U8), group_count=(2, I32), w=((2, 32, 16), U8),
                                             weight_scale=((2, 2, 1), F32), token_scale=(4, F32), out=(4 * 128, U8),
                                             workspace=(4 * 4 * 16, U8)),
}
NUMBERS = dict(eps=1e-6, a_row_bytes=128, rows=4, k=16, stream=0)


class Library:
    """Takes every call."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        return lambda *args: self.called.append(name) or 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(M, "_lib", lib)
    monkeypatch.setattr(M, "_raw_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    if hasattr(M, "_several_devices"):
        M._several_devices.cache_clear()
    yield lib
    if hasattr(M, "_several_devices"):
        M._several_devices.cache_clear()


def arguments(name):
    want = inspect.signature(getattr(M, name)).parameters
    got = {n: v for n, v in NUMBERS.items() if n in want}
    got.update({n: tensor(*v) for n, v in CALLS[name].items()})
    assert set(want) - set(got) <= {"token_scale_stride"}
    return got


@pytest.mark.parametrize("name", CALLS)
def test_current_device_is_taken(library, name):
    getattr(M, name)(**arguments(name))
    assert library.called == [name]


@pytest.mark.parametrize("name,which", [(n, t) for n, a in CALLS.items() for t in a])
def test_another_device_is_refused(library, name, which):
    got = arguments(name)
    got[which].at = 1
    with pytest.raises(ValueError, match=f"{which} is on another device than the current one"):
        getattr(M, name)(**got)
    assert library.called == []


def test_without_the_private_name(library, monkeypatch):
    monkeypatch.setattr(M, "_raw_device", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="x is on another device"):
        M.moe_rms_norm(**arguments("moe_rms_norm"))
