"""What the helpers of the microscaled operators refuse before they allocate or launch anything (no GPU needed)."""
import pytest
import torch

from weight_only_int4_act_amd import awq as A


def weights(K, N):
    kb, nt = -(-K // 128) * 4, -(-N // 64)
    return A.MxWeights(torch.zeros(nt, kb, 64, 16, dtype=torch.uint8), torch.zeros(nt, kb, 64, dtype=torch.uint8), None, K, N)


def acts(M, K, bits):
    codes = torch.zeros(M, K, dtype=torch.uint8).view(torch.float8_e4m3fn) if bits == 8 else \
        torch.zeros(M, K // 2, dtype=torch.uint8)
    return A.MxActs(codes, torch.zeros(M, K // 32, dtype=torch.uint8))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("K,other", [(128, 96), (96, 128), (32, 128), (1024, 992), (256, 128)])
def test_product_of_activations_and_weights_of_different_depths(K, other, bits):
    """Weights are padded to 128 channels, so that their buffers alone do not tell 96 channels from 128."""
    with pytest.raises(ValueError, match=f"{other} channels.*{K}"):
        A.mx_gemm(acts(3, other, bits), weights(K, 64))
    with pytest.raises(ValueError, match="device tensors"):
        A.mx_gemm(acts(3, K, bits), weights(K, 64))
