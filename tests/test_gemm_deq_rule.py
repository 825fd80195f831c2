"""The scaled expert product's tile rule (CPU only): every tile it can pick is compiled, and has a GPU case."""

import os
import re
import subprocess
import tempfile

import pytest

import instance_cases_deq as IC
import kernel_remarks

_DRIVER = r"""
#include <cstdio>
#include "select_layer.h"
int main() {
  int rows, groups, n;
  while (std::scanf("%d %d %d", &rows, &groups, &n) == 3)
    std::printf("%d\n", static_cast<int>(moe::select::gemm_deq_kind(rows, groups, n)));
}
"""
KINDS = ["stream16", "stream32", "tile64", "tile128", "tile256", "split16"]


def kinds(shapes):
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "driver.cpp"), os.path.join(d, "driver")
        with open(src, "w") as f:
            f.write(_DRIVER)
        subprocess.run(["g++", "-std=c++17", "-O1", f"-I{kernel_remarks.CSRC}", src, "-o", exe], check=True)
        text = "".join("%d %d %d\n" % s for s in shapes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    return [KINDS[int(v)] for v in out.split()]


def test_every_tile_has_a_gpu_case():
    assert sorted(IC.TILED) == sorted(KINDS)
    assert kinds([(rows, len(counts), n) for rows, n, counts in IC.TILED.values()]) == list(IC.TILED)


def test_rule_at_its_borders():
    big = 2 ** 31 - 1
    got = kinds([(1, 1, 1), (4, 1, 65536), (5, 1, 65536), (16 * 16, 16, 7168), (17 * 16, 16, 7168), (48 * 16, 16, 7168),
                 (49 * 16, 16, 7168), (128 * 16, 16, 7168), (129 * 16, 16, 7168), (4096, 2, 64), (big, 65536, 65536),
                 (1, 65536, 65536), (big, 1, 1)])
    assert got == ["split16", "stream16", "tile64", "tile64", "tile64", "tile64", "tile128", "tile128", "tile256",
                   "stream32", "tile256", "stream16", "tile256"]


def test_compiled_instances():
    if not kernel_remarks.hipcc_available():
        pytest.skip("hipcc not available")
    names = kernel_remarks.demangle(kernel_remarks.kernel_remarks()).values()
    stream = {m.group(1, 2, 3, 4, 5) for m in
              (re.search(r"::stream_kernel<\(moe::Out\)(\d), (\d+), 1, (\d+), (\d+), (\d+)>", s) for s in names) if m}
    tile = {m.group(1, 2, 3) for m in
            (re.search(r"::tile_kernel<\(moe::Out\)(\d), (\d+), \d+, \d+, (\w+)>", s) for s in names) if m}
    assert stream == {(o, *r) for o in "012" for r in (
        ("1", "1", "256", "4"), ("1", "4", "256", "1"), ("1", "2", "256", "2"), ("2", "4", "256", "1"),
        ("2", "4", "512", "1"))}
    assert tile == {(o, r, t) for o in "012" for r in ("64", "128", "256") for t in ("true", "false")}
