"""Batches of more tokens than one launch takes (CPU only): the parts that the router and the gradients are launched in
have fewer than 2^32 threads each."""

import os
import subprocess
import tempfile

import kernel_remarks

_DRIVER = r"""
#include <cstdio>
#include "select_layer.h"
using namespace moe::select;
int main() {
  std::printf("%d\n", router_launch_tokens());
  for (int k = 1; k <= 32; ++k) std::printf("%d\n", combine_backward_launch_tokens(k));
}
"""


def test_parts():
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "driver.cpp"), os.path.join(d, "driver")
        with open(src, "w") as f:
            f.write(_DRIVER)
        subprocess.run(["g++", "-std=c++17", "-O1", f"-I{kernel_remarks.CSRC}", src, "-o", exe], check=True)
        out = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    # a wave of 64 a token or entry, and a last workgroup of at most 512 threads that need not be full
    assert 0 < out[0] and out[0] * 64 + 512 < 2 ** 32 and out[0] + 512 < 2 ** 31
    for k, tokens in enumerate(out[1:], 1):
        assert 0 < tokens and tokens * k * 64 + 512 < 2 ** 32
