"""The largest numbers in the 8-bit cache, on the GPU: what is stored of them is finite or marks its block, and tokens that
nobody sees yet change nothing."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.attention_kernels import check as check_outputs
from tests.attention_kernels import take
from tests.fp8_util import Batch, attend, bf16, dev, f32
from tests.test_gpu_append import append, check, inputs

pytestmark = pytest.mark.gpu
LARGEST = 1.9921875 * 2.0 ** 127                        # of bf16
STORED = 1.9296875 * 2.0 ** 127                         # the largest bf16 number that rounds to 240 * 2^120


def setup(n, L, Hq, Hk, D, values, rows=None):
    """New tokens whose last, alone in its block, has `values` as first numbers of K and V of head 0."""
    B = Batch([(L, n)], Hq, Hk, D, 16, 3)
    if rows:
        take(B, rows)
    B.upload()
    x = inputs(B, 0, False)
    v = f32(x["qkv"]).reshape(B.M, Hq + 2 * Hk, D)
    v[n - 1, Hq, :len(values)] = values
    v[n - 1, Hq + Hk, :len(values)] = values
    x["qkv"] = bf16(v.reshape(B.M, -1))
    return B, x


def test_scale_bytes():
    assert O.cache_byte(STORED) == 247 and O.cache_byte(1.9375 * 2.0 ** 127) == 255 and O.cache_byte(LARGEST) == 255


@pytest.mark.parametrize("value", [LARGEST, 1.9375 * 2.0 ** 127, STORED, 1.75 * 2.0 ** 127])
def test_stored_numbers_are_finite(value):
    B, x = setup(2, 17, 2, 1, 64, [value, -value, 2.0 ** 126, 2.0 ** 127])
    q = append(B, x)
    k, v, E = B.download()
    blk = B.table[0, 1]
    # 1.75 2^127 is 448 2^(246 - 127), so the least E is 246 there, and 2^126 is 128 times that scale
    want = (247, [240, -240, 64, 128]) if value == STORED else (246, [448, -448, 128, 256]) if value < STORED else (255, [0] * 4)
    for c, e in ((k, E[blk, 0, 0]), (v, E[blk, 0, 1])):
        assert (e, O.code_value(c[blk, 0, 0, :4]).tolist()) == want
    check(B, x, q, label=value)


# (new tokens, tokens, heads of q, of the cache, rows a workgroup if not by the plan's own choice)
SHAPES = [(2, 17, 2, 1, None), (16, 17, 1, 1, None), (1000, 1009, 16, 1, None), (60, 65, 16, 1, 128), (100, 1009, 32, 2, 128),
          (60, 65, 32, 2, 256), (1000, 1009, 16, 1, 256)]


@pytest.mark.parametrize("n,L,Hq,Hk,rows", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_a_token_that_nobody_sees_yet(n, L, Hq, Hk, rows, D):
    got = []
    for value in (1.0, LARGEST, STORED):
        B, x = setup(n, L, Hq, Hk, D, [value, -value], rows)
        append(B, x)
        q = dev(B.queries())
        got.append(attend(B, q)[:n - 1])
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("n,L,Hq,Hk,rows", SHAPES)
def test_a_token_that_is_seen(n, L, Hq, Hk, rows):
    """Queries of zeros weigh all tokens alike: the mean with one of the largest numbers is finite, and NaN where it marks its
    block."""
    for value in (STORED, LARGEST):
        B, x = setup(n, L, Hq, Hk, 64, [value, -value], rows)
        append(B, x)
        B.k, B.v, B.E = B.download()
        q = dev(torch.zeros((B.M, Hq, 64), dtype=torch.bfloat16))
        out = attend(B, q)
        if value == STORED:
            assert torch.isfinite(out[:n].float()).all()
            check_outputs(B, rows or 16, q, out, label=(n, L))
        else:
            assert torch.isnan(out[n - 1, :Hq // Hk]).all() and torch.isfinite(out[:n - 1].float()).all()
