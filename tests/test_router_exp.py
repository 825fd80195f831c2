"""The error that include/moe_ep.h states for the choice's scores, against the library's own exponential compiled for the
CPU (its reciprocal, a hardware estimate and a Newton step, counts with 2^-44)."""

import os
import re
import subprocess
import tempfile

import pytest

import kernel_remarks

_DRIVER = r"""
#include <cmath>
#include <cstdio>
#include "exp64.h"
static double e64(double x) {
  const double n = __builtin_rint(x * moe::kLog2E);
  return std::ldexp(moe::exp_reduced(moe::kExpTerms, x, n), static_cast<int>(n));
}
int main() {
  long double up = 0, down = 0, sig = 0;  // the largest relative errors of e^x above and below it, and of 1 / (1 + e^-x)
  for (int i = -4000000; i <= 4000000; ++i) {
    const double x = i < 0 ? i * (700.0 / 4000000) : i * (104.0 / 4000000);
    const long double d = e64(x) / expl(x) - 1;
    up = fmaxl(up, d), down = fmaxl(down, -d);
    if (fabs(x) <= 104) sig = fmaxl(sig, fabsl(1.0L / (1.0L + (long double)e64(-x)) * (1.0L + expl(-(long double)x)) - 1));
  }
  std::printf("%.6Le %.6Le %.6Le\n", up, down, sig);
}
"""


@pytest.fixture(scope="module")
def errors():
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "driver.cpp"), os.path.join(d, "driver")
        with open(src, "w") as f:
            f.write(_DRIVER)
        subprocess.run(["g++", "-std=c++17", "-O2", "-mfma", "-Wno-unknown-pragmas", f"-I{kernel_remarks.CSRC}", src,
                        "-o", exe], check=True)
        return [float(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]


def test_stated_error(errors):
    up, down, sig = errors
    header = open(os.path.join(kernel_remarks.ROOT, "include", "moe_ep.h")).read()
    (bits,) = re.findall(r"binary64\s+\*\s+scores \(below 2\^-(\d+) of a score\)", header)
    stated = 2.0 ** -int(bits)
    # a softmax score is one exponential over a sum of others, which may be off to the other side
    assert max(sig, up + down) + 2.0 ** -44 < stated


def test_exponential(errors):
    """What exp64.h says of the polynomial, and that the bound is not idle."""
    assert 2.0 ** -43 < max(errors[:2]) < 2.0 ** -41
