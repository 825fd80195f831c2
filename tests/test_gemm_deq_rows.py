"""The scaled expert product's row arithmetic at the largest row counts (CPU only): a tile that starts below 2^31 may
have rows past it, which must neither be taken for an expert's nor be read from before its first row."""

import os
import re
import subprocess
import tempfile

import kernel_remarks

_DRIVER = r"""
#include <cstdio>
#include "row_range.h"
int main() {
  int row0, row_end, r;
  while (std::scanf("%d %d %d", &row0, &row_end, &r) == 3)
    std::printf("%d %d\n", moe::tile_row(row0, row_end, r), moe::tile_has_row(row0, row_end, r) ? 1 : 0);
}
"""
BIG = 2 ** 31 - 1


def test_rows_near_the_largest_int():
    cases = [(row0, row_end, r) for row0, row_end in (
        (BIG - 254, BIG), (BIG - 1, BIG), (BIG - 255, BIG - 200), (BIG - 300, BIG), (0, 1), (0, BIG), (5, 261), (7, 8))
        for r in (0, 1, 15, 31, 63, 127, 253, 254, 255)]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "driver.cpp"), os.path.join(d, "driver")
        with open(src, "w") as f:
            f.write(_DRIVER)
        # an overflow ends the program
        subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                        f"-I{kernel_remarks.CSRC}", src, "-o", exe], check=True)
        text = "".join("%d %d %d\n" % c for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    for (row0, row_end, r), line in zip(cases, out, strict=True):
        assert tuple(map(int, line.split())) == (min(row0 + r, row_end - 1), int(row0 + r < row_end)), (row0, row_end, r)


def test_the_kernels_ask_by_differences():
    """No row index of the product is formed before it is known to lie below the expert's end."""
    text = open(os.path.join(kernel_remarks.CSRC, "gemm_deq.hip")).read()
    code = re.sub(r"//.*", "", text)
    assert "row_end - 1" not in code and "< row_end" not in code and "< rs.row_end" not in code
    assert len(re.findall(r"\btile_row\(", code)) == 4 and len(re.findall(r"\btile_has_row\(", code)) == 2
