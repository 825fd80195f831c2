"""Shapes of the 8-bit float products that reach every kernel (plain data, no torch)."""

# name: (rows, n, counts) as the rule picks them (csrc/select_f8.h); counts that end inside tiles, experts without
# rows, and n that ends inside a block of 128 columns
PLAIN = {
    "split16": (50, 700, [0, 3, 5, 17, 0, 1, 2, 4, 0, 0, 9, 8, 1, 0]),
    "tile32": (200, 900, [40, 0, 33, 1, 60, 2, 3, 31, 0, 0, 9, 8, 1, 0]),
    "tile64": (900, 648, [64, 0, 65, 1, 190, 2, 63, 31] + [22] * 22),
    "tile256": (5200, 1603, [256, 2600, 0, 2300]),
}
WIDE = dict(PLAIN, tile256=(5200, 3001, [256, 2600, 0, 2300]))  # fp32 results
GATED = {  # (the rows that go through the workspace, and those that do not)
    "split16": (50, 464, [0, 3, 5, 17, 0, 1, 2, 4, 0, 0, 9, 8, 1, 0]),
    "tile32": (200, 912, [40, 0, 33, 1, 60, 2, 3, 31, 0, 0, 9, 8, 1, 0]),
    "tile64": (900, 656, [64, 0, 65, 1, 190, 2, 63, 31] + [22] * 22),
    "whole": (4200, 400, [256, 2100, 0, 1800]),
}
