"""The router's shape rule (CPU only): what it picks is compiled, holds the experts and entries, and has a GPU case."""

import os
import re
import subprocess
import tempfile

import pytest

import kernel_remarks

_DRIVER = r"""
#include <cstdio>
#include "select_layer.h"
using namespace moe::select;
int main() {
  for (const RouterShape s : kRouterShapes) std::printf("%d %d ", s.lanes, s.vpl);
  std::printf("\n");
  int bs, experts, topk;
  while (std::scanf("%d %d %d", &bs, &experts, &topk) == 3) {
    const RouterShape s = router_shape(bs, experts, topk);
    std::printf("%d %d\n", s.lanes, s.vpl);
  }
}
"""


@pytest.fixture(scope="module")
def pick():
    """Queries [(bs, E, k)] -> (table of shapes, shape of each query)."""
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "driver.cpp"), os.path.join(d, "driver")
        with open(src, "w") as f:
            f.write(_DRIVER)
        subprocess.run(["g++", "-std=c++17", "-O1", f"-I{kernel_remarks.CSRC}", src, "-o", exe], check=True)

        def run(queries):
            text = "".join("%d %d %d\n" % q for q in queries)
            lines = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
            table = list(map(int, lines[0].split()))
            return list(zip(table[::2], table[1::2])), [tuple(map(int, s.split())) for s in lines[1:]]

        yield run


def gpu_cases(name):
    """The (E, k) lists of the GPU tests, read as text (the file itself needs torch's GPU)."""
    text = open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "test_gpu_route.py")).read()
    body = re.search(rf"^{name} = \[(.*?)^\]|^{name} = \[(.*?)\]\n", text, re.S | re.M)
    return [tuple(map(int, re.findall(r"\d+", t)[:3])) for t in re.findall(r"\(([^()]*)\)", body.group(1) or body.group(2))]


def test_shapes_hold_their_call(pick):
    queries = [(bs, e, k) for bs in (1, 2047, 2048, 16384, 2 ** 26) for e in (1, 2, 16, 17, 64, 65, 255, 256, 257, 1024, 2048)
               for k in (1, 8, 16, 17, 32) if k <= e]
    table, got = pick(queries)
    for (bs, e, k), s in zip(queries, got):
        assert s in table and s[0] * s[1] >= e and s[0] >= k
        assert s[0] == 64 or bs >= 2048


def test_every_shape_is_compiled_and_has_a_gpu_case(pick):
    small = [(bs, e, k) for bs, e, k in gpu_cases("SHAPES")]
    large = [(4101, e, k) for e, k, _ in gpu_cases("LARGE")]
    table, got = pick(small + large)
    assert set(got) == set(table)
    if not kernel_remarks.hipcc_available():
        pytest.skip("hipcc not available")
    names = kernel_remarks.demangle(kernel_remarks.kernel_remarks()).values()
    for kernel in ("route_kernel", "route_backward_kernel"):
        have = {m.groups() for m in (re.search(rf"::{kernel}<(\w+), (\d+), (\d+)>", s) for s in names) if m}
        assert have == {(sig, str(lanes), str(v)) for sig in ("true", "false") for lanes, v in table}, kernel
