"""Attention's scale at the ends of its range, on the GPU: the block's scale times the call's may pass float32's range although
no score does."""
import pytest
import torch

from tests.attention_kernels import check, take
from tests.fp8_util import Batch, attend, dev

pytestmark = pytest.mark.gpu
Hq, Hk = 16, 1
SHAPES = [(16, 1, 200), (128, 60, 70), (256, 60, 70), (128, 90, 600)]    # rows a workgroup, new tokens, tokens


@pytest.mark.parametrize("rows,n,L", SHAPES)
@pytest.mark.parametrize("scale", [1e3, -1e30, 2.3e38])
def test_queries_of_zeros_under_large_scales(rows, n, L, scale):
    """All scores are zero."""
    B = take(Batch([(L, n)], Hq, Hk, 64, 16, 1), rows)
    B.E[:, :, 0] = 247
    B.k[(B.k & 127) > 0x77] = 0x77                       # 240 at most, as the append stores
    B.upload()
    q = dev(torch.zeros((B.M, Hq, 64), dtype=torch.bfloat16))
    check(B, rows, q, attend(B, q, scale=scale), scale=0.0, label=(n, scale))


@pytest.mark.parametrize("rows,n,L", SHAPES)
@pytest.mark.parametrize("E,size,scale", [(247, 2.0 ** -60, 2.0 ** -70), (240, 2.0 ** -120, 2.0 ** 8), (0, 2.0 ** 60, 2.0 ** 60),
                                          (20, 2.0 ** 97, 0.125)])
def test_scores_of_ordinary_size_from_numbers_that_are_not(rows, n, L, E, size, scale):
    B = take(Batch([(L, n)], Hq, Hk, 64, 16, 2), rows)
    B.E[:, :, 0] = E
    B.k[(B.k & 127) > 0x77] = 0x77
    if E == 0:
        B.k[(B.k & 127) < 0x20] = 0x20                   # 2^-3: its step and those above are 2^-6 or more, times 2^-127
    B.upload()
    q = dev(B.queries(size))
    check(B, rows, q, attend(B, q, scale=scale), scale=scale, label=(n, E))


@pytest.mark.parametrize("rows,n,L", SHAPES)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_scale_of_zero_and_a_query_that_is_no_number(rows, n, L, bad):
    """0 times it is NaN: its row, and no other."""
    B = take(Batch([(L, n)], Hq, Hk, 64, 16, 3), rows)
    B.upload()
    q = dev(B.queries())
    clean = attend(B, q, scale=0.0)
    check(B, rows, q, clean, scale=0.0, label=n)
    q[n - 1, Hq - 1, 5] = bad
    got = attend(B, q, scale=0.0)
    assert torch.isnan(got[n - 1, Hq - 1]).all()
    got[n - 1, Hq - 1] = clean[n - 1, Hq - 1]
    assert torch.equal(got, clean)
