"""Calls (sequences, new tokens, tokens, heads of q, heads of the cache, numbers of a head, tokens of a block) that together
reach every kernel of the attention over the cache: 16, 128 and 256 rows a workgroup, the tokens in one piece and in slices.
tests/test_attention_plan_paths.py holds the list to that."""
CASES = [
    # 16 rows, in one piece and in slices
    (7, 1, 2, 12, 4, 64, 128), (1, 32, 44, 12, 4, 128, 128), (2, 14, 785, 16, 1, 64, 64), (4, 2, 699, 16, 1, 128, 16),
    # 128 rows
    (27, 50, 54, 8, 2, 64, 64), (10, 164, 200, 16, 1, 128, 64), (1, 155, 2500, 16, 1, 64, 64), (1, 128, 1989, 16, 1, 128, 64),
    # 256 rows
    (30, 253, 1807, 16, 1, 128, 128), (1, 1396, 3002, 32, 8, 64, 32), (3, 910, 2600, 16, 1, 128, 128),
]
