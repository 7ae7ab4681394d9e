"""Sizes (M, K, N), each with 8- and 4-bit activations, that together reach every kernel of the MX product: the
register kernel with one to four fragments of 16 rows and tiles of 64, 128 and 256 rows, with K in one piece and cut
into slices, tiles also with K a multiple of 128 and not.  tests/test_mx_plan_paths.py holds the list to that."""
CASES = [
    # register kernel, K in one piece and in slices
    (5, 96, 72), (20, 352, 328), (40, 512, 264), (60, 224, 200),
    (12, 5216, 208), (30, 4256, 216), (46, 3968, 208), (55, 3712, 4544), (50, 13056, 264), (63, 4544, 2984),
    # tiles of 64 rows
    (70, 96, 136), (75, 128, 248), (100, 2208, 264), (100, 2304, 264),
    # of 128
    (2390, 1504, 1560), (2390, 512, 1560), (1260, 11200, 1712), (1408, 11264, 1360),
    # of 256
    (1576, 736, 6776), (1576, 1024, 6776), (1400, 15328, 3040), (1171, 16256, 3376),
]
