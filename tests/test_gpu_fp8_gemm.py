"""The product of 8-bit groups of 128 on the GPU against float64."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.fp8_util import A, DEV, F8, check_product, dev, f32, product, random_acts, random_weights, rows, u8

pytestmark = pytest.mark.gpu

SIZES = [(1, 16, 8), (1, 128, 64), (1, 8192, 1024), (2, 4112, 200), (5, 2080, 136), (13, 8192, 520), (16, 144, 8),
         (17, 512, 264), (31, 1040, 72), (32, 4096, 512), (33, 272, 72), (48, 1024, 128), (64, 640, 256), (65, 144, 328),
         (100, 400, 136), (128, 1024, 512), (129, 128, 256), (200, 2048, 264), (257, 1040, 384), (300, 16, 520),
         (512, 1536, 768), (700, 272, 1032), (1000, 4096, 256)]


@pytest.mark.parametrize("M,K,N", SIZES)
def test_random_codes(M, K, N):
    xc, xs, x = random_acts(M, K, M + K)
    wc, ws, w = random_weights(K, N, K + N)
    Y = product(xc, xs, wc, ws, N)
    check_product(Y, x, w, (M, K, N))


@pytest.mark.parametrize("M,K,N", [(1, 8192, 10240), (13, 5120, 13824), (257, 5120, 13824), (1024, 8192, 4096)])
def test_layers(M, K, N):
    """Quantized normal activations and weights at layer sizes, whole results against float64 on the device."""
    X = dev(rows(M, K, 1))
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    W = (torch.randn(K, N, generator=g, device=DEV) / K ** 0.5).to(torch.bfloat16)
    a, q = A.fp8_quantize(X), A.fp8_pack(W)
    Y = A.fp8_gemm(a, q)
    torch.cuda.synchronize()
    x = a.codes.double() * a.scales.double().repeat_interleave(128, 1)[:, :K]
    c = q.codes.double().view(-1, q.codes.shape[1], 4, 2, 4, 16, 16).permute(1, 3, 4, 6, 0, 2, 5)
    w = c.reshape(q.codes.shape[1] * 128, -1)[:K, :N]
    w = w * q.scales.double().t().repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]
    check_product(Y, x, w, (M, K, N))


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_marked_groups(M):
    K, N = 656, 200
    xc, xs, x = random_acts(M, K, 1)
    wc, ws, w = random_weights(K, N, 2)
    xs[M // 2, 3], ws[1, 5] = float("nan"), float("nan")
    x[M // 2, 384:512], w[640:656, 128:] = np.nan, np.nan
    Y = product(xc, xs, wc, ws, N)
    check_product(Y, x, w, M)


def test_zero_scales_and_large_ones():
    M, K, N = 40, 256, 64
    xc, xs, x = random_acts(M, K, 3)
    wc, ws, w = random_weights(K, N, 4)
    f = torch.exp2(torch.arange(M, dtype=torch.float32, device=DEV) * 4 - 100)[:, None]
    f[0] = 0
    Y = product(xc, xs * f, wc, ws, N)
    check_product(Y, x * f.double().cpu().numpy(), w, "scales")


def test_one_workspace_for_all_and_rows_behind():
    """Different shapes in turn, and the other products, over one workspace; what lies behind Y stays."""
    sizes = [(1, 8192, 1024), (5, 2080, 136), (200, 2048, 264), (33, 4096, 72), (16, 8192, 64)]
    ws = A.workspace(max(max(A.awq_fp8_gemm_workspace_size(*s) for s in sizes), 1 << 22), DEV)
    for rep in range(2):
        for M, K, N in sizes:
            xc, xs, x = random_acts(M, K, rep + M)
            wc, wsc, w = random_weights(K, N, rep + N)
            buf = torch.full((M * N + 512,), 7.0, dtype=torch.bfloat16, device=DEV)
            A.awq_fp8_gemm(xc, xs, wc, wsc, buf[:M * N].view(M, N), ws)
            torch.cuda.synchronize()
            check_product(buf[:M * N].view(M, N), x, w, (M, K, N))
            assert (buf[M * N:] == 7).all()
            assert not ws[:65536].any()


def test_repeated_calls_are_bit_identical():
    for M, K, N in ((1, 8192, 1024), (100, 4096, 512)):
        xc, xs, _ = random_acts(M, K, 5)
        wc, ws, _ = random_weights(K, N, 6)
        first = product(xc, xs, wc, ws, N)
        for _ in range(4):
            assert torch.equal(product(xc, xs, wc, ws, N), first)
