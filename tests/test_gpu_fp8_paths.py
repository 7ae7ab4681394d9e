"""Every kernel of the product with scales per 128 on the GPU, against float64 on the device: the cases of
tests/fp8_paths.py."""
import pytest
import torch

from tests.fp8_paths import CASES
from tests.fp8_util import DEV, check_product, product, random_acts, random_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", CASES)
def test_every_kernel(M, K, N):
    xc, xs, x = random_acts(M, K, M)
    wc, ws, w = random_weights(K, N, N)
    Y = product(xc, xs, wc, ws, N)
    check_product(Y, torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV), (M, K, N))
    # a NaN in one group spoils one row, also where K is cut
    xs[M // 2, (K - 1) // 256] = float("nan")
    Z = product(xc, xs, wc, ws, N)
    assert torch.isnan(Z[M // 2]).all()
    Z[M // 2] = Y[M // 2]
    assert torch.equal(Z, Y)
