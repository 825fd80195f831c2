"""The binding's stream lookup (CPU only): it imports and falls back to torch's public call where torch has not the two
private functions that it takes for speed."""

import os
import subprocess
import sys
import types

import pytest
import torch

import combine_moe_layout_03_amd as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("_cuda_getCurrentRawStream", "_cuda_getDevice")


@pytest.mark.parametrize("missing", [NAMES, NAMES[:1], NAMES[1:]], ids=lambda n: "+".join(n))
def test_imports_without_the_private_names(missing):
    code = ("import torch, types\n"
            f"for n in {missing!r}:\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import combine_moe_layout_03_amd as M\n"
            "torch.cuda.current_stream = lambda: types.SimpleNamespace(cuda_stream=77)\n"
            "assert M._stream(None) == 77 and M._stream(5) == 5\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


def test_takes_them_where_they_are(monkeypatch):
    monkeypatch.setattr(M, "_raw_device", lambda: 3)
    monkeypatch.setattr(M, "_raw_stream", lambda device: 40 + device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert M._stream(None) == 43
