"""Sizes that reach each tile of the products grouped by expert, with groups whose last
tile holds few, a quarter's, half's and nearly a whole tile's rows, and numbers of K steps
around those that are on their way at once: test_grouped_forms.py holds them against the
plan, test_gpu_grouped_forms.py runs them."""

# rows of a tile: groups' sizes, columns (plain, gated)
TILES = {
    64: ([64, 0, 1, 63, 65, 130], 70, 35),
    128: ([128, 1, 0, 64, 65, 100, 127, 30, 129], 7297, 3651),
    256: ([256, 1, 64, 65, 0, 128, 129, 255, 300, 512], 6145, 3100),
}
DEEP = (136, 256, 264, 552, 2808)                              # 16-bit K of 3, 4, 5, 9 and 44 steps
DEEP8 = (288, 512, 544, 1056, 2848)                            # 8-bit K of 3, 4, 5, 9 and 23


def all_cases():
    """(kind, rows of a tile, K, gated, gathered)"""
    for kind in ("bf16", "fp16", "row", "mx"):
        for tile in TILES:
            if tile == 256 and kind in ("row", "mx"):          # (exact 8-bit products have none)
                continue
            for i, K in enumerate(DEEP8 if kind in ("row", "mx") else DEEP):
                for gated in (False, True):
                    yield kind, tile, K, gated, (i + gated) % 2 == 0
