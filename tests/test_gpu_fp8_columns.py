"""Packed weights of any number of columns in the product, which takes multiples of 8, on the GPU: they are those of the next
multiple with columns of zeros."""
import numpy as np
import pytest
import torch

from tests.fp8_util import A, bf16, dev, u8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("K,N", [(272, 1), (400, 257), (1040, 63), (128, 515)])
def test_weights_of_any_number_of_columns(M, K, N):
    rng = np.random.default_rng(N)
    x, w = (dev(bf16(rng.standard_normal(s).astype(np.float32))) for s in ((M, K), (K, N)))
    up = -(-N // 8) * 8
    q, wide = A.fp8_pack(w), A.fp8_pack(torch.nn.functional.pad(w, (0, up - N)).contiguous())
    assert np.array_equal(u8(q.codes), u8(wide.codes)) and torch.equal(q.scales, wide.scales)
    a = A.fp8_quantize(x)
    Y = A.fp8_gemm(a, A.Fp8Weights(q.codes, q.scales, K, up))
    assert torch.equal(Y, A.fp8_gemm(a, wide)) and not Y[:, N:].any() and Y[:, :N].any(0).all()
