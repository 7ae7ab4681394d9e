"""What holds for every call of the attention, in each of its kernels (16, 128 and 256 rows a workgroup, the last two reached by
tables wider than the sequences): masks, missing and marked blocks, scores past 2^31, scales of calls and blocks, rows that
depend on nothing but themselves."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.attention_kernels import HEADS, check, take
from tests.fp8_util import A, Batch, attend, dev, f32

pytestmark = pytest.mark.gpu
ROWS = [16, 128, 256]


def most(rows, n):
    """New tokens: n where the kernel takes them."""
    return 1 if rows == 16 else n


def batch(rows, lengths, heads, D, T, seed=0):
    return take(Batch([(L, most(rows, n)) for L, n in lengths], *heads, D, T, seed), rows)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("D,T", [(64, 16), (64, 128), (128, 16), (128, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(rows, heads, D, T, causal):
    for lengths in ([(1, 1), (17, 17), (300, 3)], [(64, 64), (65, 7), (1, 1)], [(127, 1), (128, 100), (129, 9)], [(700, 90)],
                    [(513, 40), (33, 16)]):
        B = batch(rows, lengths, heads, D, T, len(lengths))
        B.upload()
        q = dev(B.queries())
        check(B, rows, q, attend(B, q, causal), causal, label=(lengths, causal))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D", [64, 128])
def test_missing_and_marked_blocks(rows, D):
    n = most(rows, 90)
    B = batch(rows, [(400, n), (170, n), (310, n)], HEADS[1], D, 16, 3)
    B.table[0, 2], B.table[0, 15], B.table[0, 23], B.table[1, :] = -1, B.blocks, np.iinfo(np.int32).min, -5
    if rows == 16:
        marks = {0: 64, 1: 300}                         # head of the cache: its first marked token
    else:
        marks = {0: 240, 1: 288}
    for (h, first), i in zip(marks.items(), (0, 1)):
        B.E[B.table[2, first // 16], h, i] = 255
    B.upload()
    q = dev(B.queries())
    for causal in (True, False):
        out = attend(B, q, causal)
        assert not out[n:2 * n].any()
        y, pos = f32(out)[2 * n:3 * n], np.arange(310 - n, 310)
        for h in range(32):
            bad = pos >= marks[h // 16] // 16 * 16 if causal else np.ones(n, bool)
            assert np.isnan(y[bad, h]).all() and not np.isnan(y[~bad, h]).any(), (causal, h)
        only = Batch([(400, n), (0, n), (0, n)], 32, 2, D, 16, 3)
        only.__dict__.update({k: v for k, v in B.__dict__.items() if k != "lengths"})
        out[n:3 * n] = 0
        check(only, rows, q, out, causal, label=("missing", causal))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("size", [2.0 ** 40, -2.0 ** 40, 2.0 ** 90])
def test_scores_past_2_to_the_31(rows, size):
    """Scores that lie further apart than any exponent: the output is V of the largest, exactly."""
    n = most(rows, 100)
    B = batch(rows, [(100, n)], HEADS[1], 64, 16, 4)
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


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D", [64, 128])
def test_a_row_is_spoiled_by_its_own_query_alone(rows, D):
    n = most(rows, 90)
    B = batch(rows, [(150, n)], HEADS[0], D, 32, 5)
    B.upload()
    q0 = dev(B.queries())
    clean = attend(B, q0)
    r = n // 3
    for bad in (float("inf"), float("-inf"), float("nan")):
        q = q0.clone()
        q[r, 5, 7] = bad
        got = attend(B, q)
        assert torch.isnan(got[r, 5]).all(), bad
        got[r, 5] = clean[r, 5]
        assert torch.equal(got, clean), bad


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("L", [150, 3000])                # 3000: in slices
def test_a_row_does_not_depend_on_the_numbers_of_others(rows, L):
    n = most(rows, 90)
    B = batch(rows, [(L, n)], HEADS[0], 128, 16, 6)
    B.upload()
    q0 = dev(B.queries())
    clean = attend(B, q0)
    for size in (2.0 ** -10, 30.0, 2.0 ** 50):            # small, beyond the running maximum, past 2^31
        q = q0.clone()
        q[n // 3, 3:6] *= size
        q[n - 1, 12] *= -size
        got = attend(B, q)
        got[n // 3, 3:6], got[n - 1, 12] = clean[n // 3, 3:6], clean[n - 1, 12]
        assert torch.equal(got, clean), size


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_scores(rows, D):
    """Large, small, zero and negative scales: exponents far apart, and all equal."""
    for scale, size in ((1.0, 4.0), (8.0, 8.0), (0.0, 1.0), (-0.1, 1.0), (1e-6, 1.0)):
        B = batch(rows, [(333, 60), (50, 50)], HEADS[0], D, 32, 7)
        B.upload()
        q = dev(B.queries(size))
        check(B, rows, q, attend(B, q, scale=scale), scale=scale, label=(scale, size))


@pytest.mark.parametrize("rows", ROWS)
def test_blocks_of_very_different_scales(rows):
    B = batch(rows, [(500, 90)], HEADS[1], 64, 16, 8)
    B.E[:, :, 0] = B.rng.integers(100, 124, B.E.shape[:2])
    B.E[:, :, 1] = B.rng.integers(20, 200, B.E.shape[:2])
    B.E[B.table[0, 3]] = 0
    B.upload()
    q = dev(B.queries())
    check(B, rows, q, attend(B, q), label="scales")


@pytest.mark.parametrize("rows", [128, 256])
def test_one_workspace_and_rows_past_the_last_sequence(rows):
    """Long and short sequences in turn over one workspace; rows that no sequence has stay."""
    ws = A.workspace(1 << 27, "cuda:0")
    for rep in range(2):
        for lengths in ([(3000, 60)], [(200, 90), (9, 9)], [(1500, 3), (700, 70)]):
            B = batch(rows, lengths, HEADS[0], 64, 64, rep)
            B.upload()
            q = dev(B.queries())
            assert A.awq_attention_workspace_size(B.M, len(lengths), B.max_q, B.Hq, B.Hk, 64) <= ws.numel()
            out = attend(B, q, ws=ws)
            check(B, rows, q, out, label=(rep, lengths))
            assert torch.equal(out, attend(B, q, ws=ws)) and not ws[:65536].any()
