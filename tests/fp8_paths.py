"""Sizes (M, K, N) that together reach every kernel of the product with scales per 128: the register kernel with one, two and
four fragments of 16 rows and tiles of 64, 128 and 256 rows, with K in one piece and cut into slices, tiles also with K a
multiple of 128 and not.  tests/test_fp8_plan_paths.py holds the list to that."""
CASES = [
    # register kernel, K in one piece and in slices
    (5, 240, 72), (24, 112, 80), (303, 400, 840), (3, 8336, 40), (30, 1408, 520), (223, 12880, 168),
    # tiles of 64 rows
    (122, 48, 15816), (395, 128, 3184), (65, 4240, 224), (294, 5120, 832),
    # of 128
    (808, 144, 5984), (976, 256, 4824), (379, 9120, 808), (352, 4864, 1584),
    # of 256
    (924, 144, 10104), (700, 256, 13320), (668, 14992, 5416), (490, 17920, 8576),
]
