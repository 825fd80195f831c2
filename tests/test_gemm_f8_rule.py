"""The rules of the 8-bit float products and of the norm (CPU only): every kernel they can pick is compiled, has a GPU
case, and keeps to what the kernels assume."""

import os
import re
import subprocess
import tempfile

import pytest

import instance_cases_f8 as IC
import kernel_remarks

_DRIVER = r"""
#include <cstdio>
#include "select_f8.h"
#include "select_norm.h"
using namespace moe::select;
int main() {
  char what;
  int a, b, c;
  while (std::scanf(" %c %d %d %d", &what, &a, &b, &c) == 4) {
    if (what == 'p') std::printf("%d\n", static_cast<int>(gemm_f8_kind(a, b, c, false)));
    if (what == 'w') std::printf("%d\n", static_cast<int>(gemm_f8_kind(a, b, c, true)));
    if (what == 'g') std::printf("%d\n", gemm_f8_act(a, b, c) ? static_cast<int>(gemm_f8_act_kind(a, b, c)) : 9);
    if (what == 'n') {
      const NormShape s = norm_shape(b);
      std::printf("%d %d %d %d\n", s.chunks, s.waves, norm_backward_rows(s.waves), norm_backward_parts(a, b));
    }
  }
}
"""
KINDS = {0: "split16", 1: "tile32", 2: "tile64", 3: "tile256", 9: "whole"}


def answers(lines):
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "driver.cpp"), os.path.join(d, "driver")
        with open(src, "w") as f:
            f.write(_DRIVER)
        subprocess.run(["g++", "-std=c++17", "-O1", f"-I{kernel_remarks.CSRC}", src, "-o", exe], check=True)
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
    return [tuple(int(v) for v in line.split()) for line in out.splitlines()]


def kinds(what, shapes):
    return [KINDS[v[0]] for v in answers(["%s %d %d %d" % (what, *s) for s in shapes])]


def test_every_kernel_has_a_gpu_case():
    assert kinds("p", [(r, len(c), n) for r, n, c in IC.PLAIN.values()]) == list(IC.PLAIN)
    assert kinds("w", [(r, len(c), n) for r, n, c in IC.WIDE.values()]) == list(IC.WIDE)
    assert kinds("g", [(r, len(c), n) for r, n, c in IC.GATED.values()]) == list(IC.GATED)
    assert set(IC.PLAIN) == {"split16", "tile32", "tile64", "tile256"}
    assert set(IC.WIDE) == set(IC.PLAIN)
    assert set(IC.GATED) == {"split16", "tile32", "tile64", "whole"}


def test_rules_at_their_borders():
    big = 2 ** 31 - 1
    assert kinds("p", [(1, 1, 1), (16, 1, 8192), (17, 1, 16384), (16, 16, 7168), (256, 16, 7168), (257, 16, 7168),
                       (128 * 16, 16, 7168), (129 * 16, 16, 7168), (4096, 2, 64), (big, 65536, 65536), (1, 65536, 65536),
                       (big, 1, 1)]) == [
        "split16", "split16", "tile64", "tile32", "tile32", "tile64", "tile64", "tile256", "tile64", "tile256", "tile32",
        "tile256"]
    assert kinds("w", [(129 * 16, 16, 7168), (8000, 8, 1024), (16384, 4, 2048), (big, 65536, 65536)]) == [
        "tile256", "tile64", "tile256", "tile256"]
    assert kinds("g", [(1, 1, 16), (8, 8, 2048), (8, 8, 1536), (256, 16, 2048), (257, 16, 2048), (4096, 64, 2048),
                       (4096, 16, 2048), (4096, 1, 64), (4097, 1, 16), (big, 65536, 32768)]) == [
        "split16", "tile32", "split16", "tile32", "tile64", "tile64", "whole", "tile64", "whole", "whole"]


def test_norm_shapes():
    """At most eight waves, a chunk for every eight columns, parts within the workspace's bound."""
    widths = list(range(8, 16385, 8))
    for h, (chunks, waves, rows, parts) in zip(widths, answers(["n %d %d 0" % (2 ** 31 - 1, h) for h in widths])):
        assert chunks in (1, 2, 4) and 1 <= waves <= 8 and 64 * chunks * waves * 8 >= h
        assert (chunks != 1 or waves == 1) and (chunks != 4 or waves > 4)
        assert 1 <= rows * waves <= 8 and parts == 256 and (rows == 1 or h <= 4096)
    assert [v[3] for v in answers(["n 0 64 0", "n 1 64 0", "n 8 64 0", "n 9 64 0", "n 300 7168 0", "n 3 7168 0"])] == [
        0, 1, 1, 2, 256, 3]


def test_compiled_instances():
    if not kernel_remarks.hipcc_available():
        pytest.skip("hipcc not available")
    names = list(kernel_remarks.demangle(kernel_remarks.kernel_remarks()).values())

    def found(pattern):
        return {m.groups() for m in (re.search(pattern, s) for s in names) if m}

    assert found(r"::split_f8_kernel<\(moe::Form\)(\d)>") == {(f,) for f in "0124"}
    ring = found(r"::ring_f8_kernel<\(moe::Form\)(\d), (\w+), (\d+), (\d+), \d+, \d+, (\w+)>")
    tails = ("true", "false")
    assert ring == {(f, "true" if f in "24" else "false", m, "128", t) for f in "0124" for m in ("32", "64")
                    for t in tails} | {("2", "true", "256", "128", t) for t in tails} | {
                        ("3", "true", "128", "256", t) for t in tails}
    assert found(r"::tile_f8_kernel<\(moe::Form\)(\d), (\d+), (\d+), \d+, \d+, (\w+)>") == {
        (f, "256", "256", t) for f in "01" for t in tails}
    shapes = {("1", "true", "false"), ("2", "true", "false"), ("2", "false", "false"), ("2", "false", "true"),
              ("4", "false", "false"), ("4", "false", "true")}
    assert found(r"::rms_norm_kernel<\(moe::Out\)(\d), (\d), (\w+), (\w+)>") == {(t, *s) for t in "012" for s in shapes}
    assert found(r"::rms_norm_backward_kernel<\(moe::Out\)(\d), \(moe::Out\)(\d), (\d), (\w+), (\w+)>") == {
        (t, g, *s) for t in "012" for g in "012" for s in shapes}
