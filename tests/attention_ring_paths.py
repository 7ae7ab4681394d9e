"""Calls (sequences, new tokens, tokens, heads of q, heads of the cache, numbers of a head, tokens of a block) in which the
attention's tiles, of 128 and of 256 rows at both sizes of a head, in one piece and in slices where the plan has both, fill each
of their two stages twice at least.  tests/test_attention_ring_paths.py holds the list to that."""
CASES = [(12, 200, 768, 16, 2, 64, 64), (12, 200, 768, 16, 2, 128, 16), (1, 600, 4096, 16, 1, 128, 128),
         (1, 155, 2500, 16, 1, 64, 32), (1, 1396, 3002, 32, 8, 64, 32), (3, 910, 2600, 16, 1, 128, 128),
         (30, 253, 1807, 16, 1, 128, 128)]
