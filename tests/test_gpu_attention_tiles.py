"""Attention of many rows per head of the cache: the tiles of 128 and of 256 rows and their joined slices, at the numbers
of rows where the kernels change, with every block size, and scores past 2^31."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.fp8_util import Batch, attend, check_attention, dev, f32

pytestmark = pytest.mark.gpu


def run(lengths, Hq, Hk, D, T, seed=0, causal=True):
    B = Batch(lengths, Hq, Hk, D, T, seed)
    B.upload()
    q = dev(B.queries())
    check_attention(B, q, attend(B, q, causal), causal, label=(lengths, Hq, Hk, D, T, causal))


@pytest.mark.parametrize("n", [8, 9, 32, 33, 64, 255, 256, 257])
@pytest.mark.parametrize("D", [64, 128])
def test_where_the_kernels_change(n, D):
    run([(n + 50, n), (n, n), (3, 1)], 4, 1, D, 32, n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_256_rows(D, T, causal):
    run([(300, 300), (700, 270), (5, 5), (33, 1), (129, 128)], 8, 2, D, T, 1, causal)


@pytest.mark.parametrize("lengths", [[(20011, 40)], [(9000, 300), (100, 20)], [(5000, 2), (4099, 12)]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_slices(lengths, D, causal):
    run(lengths, 8, 2, D, 16, 2, causal)


def test_missing_and_marked_blocks_of_256_rows():
    n = 300
    B = Batch([(400, n), (600, n), (310, n)], 8, 2, 128, 16, 3)
    B.table[0, 2], B.table[0, 15], B.table[1, :] = -1, B.blocks, -5
    B.E[B.table[2, 4], 0, 0] = B.E[B.table[2, 9], 1, 1] = 255     # tokens 64 .. and 144 ..
    B.upload()
    q = dev(B.queries())
    for causal in (True, False):
        out = attend(B, q, causal)
        assert not out[n:2 * n].any()
        y, pos = f32(out)[2 * n:3 * n], np.arange(310 - n, 310)
        for h in range(8):
            bad = pos >= (64 if h < 4 else 144) if causal else np.ones(n, bool)
            assert np.isnan(y[bad, h]).all() and not np.isnan(y[~bad, h]).any(), (causal, h)
        only = Batch([(400, n), (0, n), (0, n)], 8, 2, 128, 16, 3)
        only.__dict__.update({k: v for k, v in B.__dict__.items() if k != "lengths"})
        out[n:3 * n] = 0
        check_attention(only, q, out, causal, label=("missing", causal))


@pytest.mark.parametrize("n", [1, 30, 100])
@pytest.mark.parametrize("size", [2.0 ** 40, -2.0 ** 40, 2.0 ** 90])
def test_scores_past_2_to_the_31(n, size):
    """Scores that lie further apart than any exponent: the output is V of the largest, exactly."""
    B = Batch([(100, n)], 32, 2, 64, 16, 4)
    order = B.rng.permutation(100) + 1                    # codes 1 .. 100 of number 0, ascending values
    B.k[:], B.E[:] = 0, 127
    for t in range(100):
        B.k[B.table[0, t // 16], :, t % 16, 0] = order[t]
    B.upload()
    x = torch.zeros((B.M, 32, 64), dtype=torch.bfloat16)
    x[:, :, 0] = size
    q = dev(x)
    value = O.code_value(order.astype(np.uint8)) * np.sign(size)
    _, v = B.cached(0)
    for causal in (True, False):
        y = f32(attend(B, q, causal))[:n]
        for r in range(n):
            best = int(np.argmax(value[:100 - n + r + 1 if causal else 100]))
            assert np.array_equal(y[r], np.repeat(v[best], 16, axis=0)), (causal, r)


@pytest.mark.parametrize("n", [3, 50, 100])
def test_an_infinite_query_spoils_its_own_row_only(n):
    B = Batch([(150, n)], 32, 2, 64, 32, 5)
    B.upload()
    x = B.queries()
    q0 = dev(x)
    clean = attend(B, q0)
    for bad in (float("inf"), float("-inf"), float("nan")):
        q = q0.clone()
        q[1, 5, 7] = bad
        got = attend(B, q)
        assert torch.isnan(got[1, 5]).all(), bad
        got[1, 5] = clean[1, 5]
        assert torch.equal(got, clean), bad


@pytest.mark.parametrize("n", [3, 50, 100])
def test_a_row_does_not_depend_on_the_numbers_of_others(n):
    B = Batch([(150, n)], 32, 2, 128, 16, 6)
    B.upload()
    q0 = dev(B.queries())
    clean = attend(B, q0)
    for size in (2.0 ** -10, 30.0, 2.0 ** 50):            # small, beyond the running maximum, past 2^31
        q = q0.clone()
        q[1, 3:6] *= size
        q[n - 1, 20] *= -size
        got = attend(B, q)
        got[1, 3:6], got[n - 1, 20] = clean[1, 3:6], clean[n - 1, 20]
        assert torch.equal(got, clean), size


@pytest.mark.parametrize("lengths", [[(130, 1), (1, 1)], [(100, 20), (40, 3)], [(292, 85), (60, 60)], [(500, 300), (3, 2)]])
@pytest.mark.parametrize("D", [64, 128])
def test_a_table_much_wider_than_the_sequences(lengths, D):
    """The width chooses the kernel and the slices; columns behind the last token are not looked at."""
    B = Batch(lengths, 8, 2, D, 32, 7)
    n, width = B.table.shape
    rest = B.rng.integers(-5, B.blocks + 5, (n, 1000)).astype(np.int32)
    rest[:, ::7] = np.iinfo(np.int32).max
    B.table = np.concatenate((B.table, rest), 1)
    for b, (L, _) in enumerate(lengths):
        B.table[b, -(-L // 32):width] = rest[b, 0]
    B.upload()
    q = dev(B.queries())
    for causal in (True, False):
        check_attention(B, q, attend(B, q, causal), causal, label=(lengths, D, causal))


@pytest.mark.parametrize("n", [1, 60])
def test_many_short_sequences_and_one_long(n):
    run([(9000, n)] + [(L, min(L, n)) for L in range(1, 60)], 8, 2, 128, 16, 8)
