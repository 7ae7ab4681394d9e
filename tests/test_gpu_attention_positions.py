"""Attention of more new tokens than a sequence has tokens, on the GPU: the rows at positions below zero are zero, causal or
not, in every kernel."""
import numpy as np
import pytest

from oracle import fp8_oracle as O
from tests.fp8_util import Batch, attend, check_attention, dev

pytestmark = pytest.mark.gpu


def test_the_oracle_gives_zeros():
    q, k = np.ones((4, 2)), np.zeros((2, 2))
    v = np.array([[1.0, 0], [3, 0]])
    assert O.attention(q, k, v, True, 1.0)[0][:, 0].tolist() == [0, 0, 1, 2]
    assert O.attention(q, k, v, False, 1.0)[0][:, 0].tolist() == [0, 0, 2, 2]


# 16, 128 and 256 rows a workgroup, also with the tokens in slices; a boundary inside a wavefront's rows and between them
@pytest.mark.parametrize("lengths", [[(3, 5)], [(1, 2), (7, 16), (60, 1)], [(40, 70), (10, 64), (64, 65)],
                                     [(200, 300), (64, 256), (300, 310)], [(700, 900)], [(1500, 1503)]])
@pytest.mark.parametrize("Hq,Hk,D,T", [(1, 1, 64, 16), (8, 2, 128, 64), (16, 1, 64, 32), (16, 1, 128, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_before_the_first_token(lengths, Hq, Hk, D, T, causal):
    B = Batch(lengths, Hq, Hk, D, T, 5)
    B.upload()
    q = dev(B.queries())
    out = attend(B, q, causal)
    for b, (L, n) in enumerate(lengths):
        assert not out[B.cu[b]:B.cu[b] + max(n - L, 0)].any(), (lengths[b], causal)
    check_attention(B, q, out, causal, label=(lengths, Hq, Hk, D, T, causal))
