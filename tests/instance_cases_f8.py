"""Shapes of the 8-bit float products that reach every kernel (plain data, no torch)."""

# name: (rows, n, counts) as the rule picks them (csrc/select_f8.h); counts that end inside tiles, experts without
# rows, and n that ends inside a block of 128 columns
PLAIN = {
    "stream32": (200, 900, [40, 0, 33, 1, 60, 2, 3, 31, 0, 0, 9, 8, 1, 0]),
}
GATED = {
    "stream32": (200, 912, [40, 0, 33, 1, 60, 2, 3, 31, 0, 0, 9, 8, 1, 0]),
}
