"""What the 8-bit float products' sums may be off by, as a whole: the norm of the
error over many results, which wrong scales, lost terms and sums in fewer bits
pass far sooner than they pass the bound of a single result.
"""

import numpy as np
import torch

import block_rows_ref as B

# What the 8-bit matrix instruction loses of normally distributed rows' results, as the header states it, twice; and
# what binary32 sums lose: the roundings of some 2000 terms add up like a walk, 2^-24 sqrt(2000) = 2.7e-6 at most.
STATED = 2 * 1.4e-5
EXACT = 2.7e-6


def rounded(v, kind):
    return torch.from_numpy(v).to(B.TYPES[kind]).double().numpy()


def check_norm(got, want, kind, off):
    """got, of a type, against want, from which the values before their rounding are off by `off` of its norm.

    A value y + d is rounded to the nearest of the type, whose distance from it is at most that of y and |d|; so got is
    at most that distance and 2 |d| from y."""
    nearest = np.linalg.norm(rounded(want, kind) - want)
    assert np.linalg.norm(got - want) <= nearest + 2 * off * np.linalg.norm(want)
