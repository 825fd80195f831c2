"""Shapes of the scaled int8 expert product that reach every tile (plain data, no torch)."""

# tile: (rows, n, counts), the tile as the launcher's rule picks it (csrc/select_layer.h, gemm_deq_kind); counts that end
# inside tiles, experts without rows, and n that ends inside a column tile
TILED = {
    "split16": (50, 700, [0, 3, 5, 17, 0, 1, 2, 4, 0, 0, 9, 8, 1, 0]),
    "stream16": (50, 1900, [0, 3, 5, 17, 0, 1, 2, 4, 0, 0, 9, 8, 1, 0]),
    "stream32": (200, 900, [40, 0, 33, 1, 60, 2, 3, 31, 0, 0, 9, 8, 1, 0]),
    "tile64": (900, 648, [64, 0, 65, 1, 190, 2, 63, 31] + [22] * 22),
    "tile128": (1800, 700, [128, 0, 129, 1, 400, 2, 127, 31] + [80] * 12),
    "tile256": (5200, 1603, [256, 2600, 0, 2300]),
}
