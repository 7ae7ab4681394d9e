"""Sizes (M, K, N) that together reach every kernel of the product with scales per 128: the register kernel with one, two and
four fragments of 16 rows and tiles of 64, 128 and 256 rows, with K in one piece and cut into slices, tiles also with K a
multiple of 128 and not.  tests/test_fp8_plan_paths.py holds the list to that."""
CASES = [
    # register kernel, K in one piece and in slices
    (5, 240, 72), (24, 112, 80), (35, 1600, 9080), (3, 8336, 40), (30, 1408, 520), (39, 2880, 4128),
    # tiles of 64 rows
    (200, 48, 1232), (104, 256, 4296), (98, 1328, 48), (130, 9600, 40),
    # of 128
    (808, 144, 5984), (976, 256, 4824), (230, 15472, 8600), (682, 16896, 2712),
    # of 256
    (924, 144, 10104), (700, 256, 13320), (656, 16192, 5408), (490, 17920, 8576),
]
