"""Attention of more new tokens than a sequence has tokens, on the GPU: the rows at positions below zero are zero, causal or
not, in every kernel."""
import numpy as np
import pytest

from oracle import fp8_oracle as O
from tests.attention_kernels import HEADS, check, take
from tests.fp8_util import Batch, attend, dev

pytestmark = pytest.mark.gpu


def test_the_oracle_gives_zeros():
    q, k = np.ones((4, 2)), np.zeros((2, 2))
    v = np.array([[1.0, 0], [3, 0]])
    assert O.attention(q, k, v, True, 1.0)[0][:, 0].tolist() == [0, 0, 1, 2]
    assert O.attention(q, k, v, False, 1.0)[0][:, 0].tolist() == [0, 0, 2, 2]


def run(B, rows, causal, label):
    B.upload()
    q = dev(B.queries())
    out = attend(B, q, causal)
    for b, (L, n) in enumerate(B.lengths):
        assert not out[B.cu[b]:B.cu[b] + max(n - L, 0)].any(), (label, B.lengths[b], causal)
    check(B, rows, q, out, causal, label=(label, causal))


# by 16 rows a workgroup; a boundary inside its rows and between them
@pytest.mark.parametrize("lengths", [[(3, 5)], [(1, 2), (7, 16), (60, 1)], [(40, 70), (10, 64), (64, 65)],
                                     [(200, 300), (64, 256), (300, 310)], [(700, 900)], [(1500, 1503)]])
@pytest.mark.parametrize("Hq,Hk,D,T", [(1, 1, 64, 16), (8, 2, 128, 64), (16, 1, 64, 32), (16, 1, 128, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_before_the_first_token(lengths, Hq, Hk, D, T, causal):
    run(Batch(lengths, Hq, Hk, D, T, 5), 16, causal, (lengths, Hq, Hk, D, T))


@pytest.mark.parametrize("rows,lengths", [(128, [(3, 5)]), (128, [(40, 70), (10, 64), (64, 65)]), (128, [(1, 90)]),
                                          (256, [(200, 300), (64, 256), (300, 310)]), (256, [(700, 900)]),
                                          (256, [(1200, 1203), (5, 9)])])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("D,T", [(64, 16), (128, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_before_the_first_token_in_tiles(rows, lengths, heads, D, T, causal):
    """Of 128 and 256 rows, also with the tokens in slices; a boundary inside a wavefront's rows and between them."""
    run(take(Batch(lengths, *heads, D, T, 5), rows), rows, causal, (rows, lengths, heads, D, T))
