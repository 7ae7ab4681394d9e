"""Attention over the 8-bit cache on the GPU against float64: lengths from zero on, heads in every grouping, ragged batches,
decode and prefill, masks, marked and missing blocks, unwritten slots."""
import numpy as np
import pytest
import torch

from tests.fp8_util import A, DEV, Batch, attend, check_attention, dev, f32

pytestmark = pytest.mark.gpu


def run(lengths, Hq, Hk, D, T, seed=0, causal=True, scale=None, size=1.0):
    B = Batch(lengths, Hq, Hk, D, T, seed)
    B.upload()
    q = dev(B.queries(size))
    out = attend(B, q, causal, scale)
    check_attention(B, q, out, causal, scale, (lengths[:4], Hq, Hk, D, T, causal))
    return B, q, out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (8, 1), (6, 2), (16, 1), (5, 1), (17, 1)])
def test_decode(D, T, Hq, Hk):
    run([(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (63, 1), (64, 1), (65, 1), (200, 1), (1031, 1), (129, 1)], Hq, Hk, D, T)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [16, 64, 128])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (8, 1), (6, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill(D, T, Hq, Hk, causal):
    run([(1, 1), (5, 5), (64, 64), (130, 130), (77, 40), (300, 33), (257, 200), (90, 2)], Hq, Hk, D, T, 1, causal)


@pytest.mark.parametrize("lengths", [[(4097, 1)], [(20011, 1), (3, 1)], [(2500, 700)], [(1500, 1500), (1, 1)], [(3000, 4)]])
@pytest.mark.parametrize("D", [64, 128])
def test_long(lengths, D):
    run(lengths, 8, 2, D, 64, 2)


def test_many_sequences():
    rng = np.random.default_rng(3)
    run([(int(L), 1) for L in rng.integers(1, 700, 200)], 4, 1, 64, 16, 3)
    run([(int(L), int(min(L, n))) for L, n in zip(rng.integers(1, 200, 60), rng.integers(1, 90, 60))], 4, 2, 128, 32, 4)


def test_rows_that_see_nothing_are_zero():
    """Length zero, fewer tokens than new ones, blocks that are missing at the front, in the middle and altogether."""
    for n in (1, 9, 150):
        B = Batch([(300, n), (40, n), (100, n), (7, n), (64, n)], 4, 2, 64, 16, n)
        B.lengths[1], B.lengths[3] = (0, n), (-3, n)
        B.table[2, :] = -1
        B.table[0, 0], B.table[0, 4], B.table[4, 1] = -1, B.blocks + 7, np.iinfo(np.int32).min
        B.upload()
        q = dev(B.queries())
        for causal in (True, False):
            out = attend(B, q, causal)
            for b in (1, 2, 3):
                assert not out[B.cu[b]:B.cu[b] + n].any(), (n, b)
            keep = B.lengths
            B.lengths = [(L if b in (0, 4) else 0, k) for b, (L, k) in enumerate(B.lengths)]
            check_attention(B, q, out, causal, label=("missing", n))
            B.lengths = keep


def test_length_past_the_table():
    B = Batch([(100, 1), (60, 60)], 4, 2, 64, 16, 5)
    B.upload()
    B.lengths = [(2 ** 31 - 1, 1), (60, 60)]
    B.d["length"][0] = 2 ** 31 - 1
    # all the table's tokens are seen, whatever the slots behind the hundredth hold: make them numbers
    B.k[(B.k & 127) == 127], B.v[(B.v & 127) == 127] = 0, 0
    B.upload()
    B.d["length"][0] = 2 ** 31 - 1
    q = dev(B.queries())
    out = attend(B, q)
    B.lengths = [(B.table.shape[1] * 16, 1), (60, 60)]
    check_attention(B, q, out, label="past the table")


@pytest.mark.parametrize("n", [1, 70])
def test_marked_blocks(n):
    """A block of scale 255 makes NaN of what is seen of it, and of nothing else."""
    B = Batch([(200, n)], 4, 2, 64, 16, 6)
    B.E[B.table[0, 11], 0, 0] = 255                       # K of tokens 176 .. 191, head 0
    B.E[B.table[0, 12], 1, 1] = 255                       # V of tokens 192 .. 199, head 1
    B.upload()
    q = dev(B.queries())
    out = f32(attend(B, q))[B.cu[0]:B.cu[0] + n]
    pos = np.arange(200 - n, 200)
    for h, first in ((0, 176), (1, 176), (2, 192), (3, 192)):
        assert np.isnan(out[pos >= first, h]).all() and not np.isnan(out[pos < first, h]).any()


@pytest.mark.parametrize("n", [1, 100])
def test_scales_of_scores(n):
    """Large, small, zero and negative scales: exponents far apart, and all equal."""
    for scale, size in ((1.0, 4.0), (8.0, 8.0), (0.0, 1.0), (-0.1, 1.0), (1e-6, 1.0)):
        run([(333, n), (50, min(n, 50))], 4, 2, 128, 32, 7, scale=scale, size=size)


@pytest.mark.parametrize("n", [1, 100])
def test_blocks_of_very_different_scales(n):
    B = Batch([(500, n)], 4, 2, 64, 16, 8)
    B.E[:, :, 0] = B.rng.integers(100, 124, B.E.shape[:2])
    B.E[:, :, 1] = B.rng.integers(20, 200, B.E.shape[:2])
    B.E[B.table[0, 3]] = 0
    B.upload()
    q = dev(B.queries())
    check_attention(B, q, attend(B, q), label="scales")


def test_one_workspace_and_repeated_calls():
    ws = A.workspace(1 << 26, DEV)
    for rep in range(3):
        for lengths, n in (([(3000, 1)], 1), ([(700, 1)] * 5, 1), ([(2000, 3), (10, 2)], 3), ([(90, 90)], 90)):
            B = Batch(lengths, 8, 2, 64, 64, rep)
            B.upload()
            q = dev(B.queries())
            assert A.awq_attention_workspace_size(B.M, len(lengths), n, 8, 2, 64) <= ws.numel()
            out = attend(B, q, ws=ws)
            check_attention(B, q, out, label=(rep, lengths))
            assert not ws[:65536].any()
            assert torch.equal(out, attend(B, q, ws=ws))


def test_rows_past_max_q_are_left_as_they_were():
    B = Batch([(100, 60), (30, 5)], 4, 2, 64, 16, 12)
    B.upload()
    q = dev(B.queries())
    out = attend(B, q, max_q=8)
    assert (out[8:60] == 7).all() and not (out[:8] == 7).any() and not (out[60:65] == 7).any()
