"""Attention of up to 16 rows per head of the cache on the GPU: p enters the second product with 16 bits, not with bf16's eight,
so that results whose terms cancel are as near as float32 sums give them."""
import numpy as np
import pytest

from oracle import fp8_oracle as O
from tests.fp8_util import H32, HBF, Batch, attend, bf16, dev, f32

pytestmark = pytest.mark.gpu


def bound(out, size, reach, D, L):
    """That of tests/fp8_util.py but for p's rounding: p's nearest bf16 number and the nearest bf16 number of what is left miss p
    by 2^-8 of 2^-8 of it at most; its sum is of the float32 numbers."""
    p = (2 * D + 4) * H32 * reach + 2 * H32
    return HBF * np.abs(out) + size * (2.0 ** -16 + 2 * p + 2 * (L + 64) * H32) + 2.0 ** -126


def batch(lengths, Hq, Hk, D):
    """Scores near zero and V of plus and minus one number, whose means cancel."""
    B = Batch(lengths, Hq, Hk, D, 16, 7)
    B.v[:] = 0x38 | B.rng.integers(0, 2, B.v.shape).astype(np.uint8) * 128
    B.E[:, :, 1] = 127
    return B, B.queries(0.1)


def results(B, q):
    """Of every row: the definition, the sum of p |v|, the reach, and what p of eight bits would give."""
    x, G = f32(q).astype(np.float64), B.Hq // B.Hk
    for b, (L, n) in enumerate(B.lengths):
        k, v = B.cached(b)
        for h in range(B.Hq):
            r = slice(B.cu[b], B.cu[b] + n)
            out, size, reach = O.attention(x[r, h], k[:, h // G], v[:, h // G], True, B.D ** -0.5)
            s = x[r, h] @ k[:, h // G].T * B.D ** -0.5
            s[np.arange(L)[None] > np.arange(L - n, L)[:, None]] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            short = f32(bf16(p)).astype(np.float64) @ v[:, h // G] / p.sum(1, keepdims=True)
            yield r, h, out, bound(out, size, reach, B.D, L), short


LENGTHS = [[(16, 1), (5, 1), (40, 2), (129, 3)], [(700, 1), (33, 2)]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (5, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_p_of_16_bits(lengths, Hq, Hk, D):
    B, q = batch(lengths, Hq, Hk, D)
    B.upload()
    y = f32(attend(B, dev(q))).astype(np.float64)
    missed = 0
    for r, h, out, allowed, short in results(B, q):
        ok = np.abs(y[r, h] - out) <= allowed
        assert ok.all(), (r, h, np.abs(y[r, h] - out)[~ok][:4], allowed[~ok][:4])
        missed += int((np.abs(short - out) > allowed).sum())
    assert missed > 10, "eight bits of p would not be told from 16"
