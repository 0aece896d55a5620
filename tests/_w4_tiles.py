"""Shapes that reach each tile of the kernel for many tokens, {16s of tokens, 64s of
weight rows}: rows that end in a wave's first 16s, in its last, and before a wave that
then has none.  Test infrastructure."""

TILES = {
    (1, 1): [(17, 4161), (49, 2049), (130, 1000)],
    (2, 1): [(33, 5500), (64, 4097), (130, 1793)],
    (1, 2): [(40, 8193), (130, 3265), (130, 3333)],
    (2, 2): [(17, 16393), (100, 4700), (130, 3585)],
    (4, 2): [(65, 10900), (130, 6529), (130, 6600)],
}
CASES = [(tile, m, n) for tile, shapes in TILES.items() for m, n in shapes]

# whole groups of 512 for two rounds of eight waves, the last of them not whole; and,
# row-major, a rest that ends inside a stretch of 128
PACKED_K, ROWS_K = 5120, {32: 5344, 16: 5328}
