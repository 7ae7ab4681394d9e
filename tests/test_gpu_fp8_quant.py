"""The 8-bit groups of 128 on the GPU against the float64 oracle: activations (with and without a gate) and weights."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from oracle.mx_oracle import gated
from tests.fp8_util import A, DEV, F8, H32, bf16, check_groups, dev, f32, rows, u8

pytestmark = pytest.mark.gpu


def extremes(x, seed):
    """Plants groups of zeros, subnormals, borders, the largest numbers, an infinity and a NaN into x [R, K] (K a multiple
    of 128)."""
    x = x.copy()
    b = x.reshape(-1, 128)
    plant = [np.zeros(128), np.full(128, -0.0), np.full(128, 2.0 ** -130), np.r_[448, np.tile([17, 19, 2.0 ** -9, 2.0 ** -10, 256, 255, -3], 18), 1],
             np.full(128, 3.3e38), np.full(128, -2.0 ** 120), np.r_[np.inf, np.ones(127)], np.r_[np.ones(127), np.nan],
             np.r_[2.0 ** 100, np.full(127, 2.0 ** -100)], np.r_[2.0 ** -111, np.full(127, 2.0 ** -118)],
             np.full(128, -2.0 ** -112)]
    for i, r in enumerate(np.random.default_rng(seed).permutation(b.shape[0])[:len(plant)]):
        b[r] = plant[i]
    return x


def check_acts(a, p, delta, label):
    K = p.shape[1]
    check_groups(u8(a.codes), a.scales.cpu().numpy(), O.scale_of, p, delta, lambda s: O.spread_rows(s, K), O.group_top(p),
                 label)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 8192), (3, 144), (5, 2064), (16, 28672), (129, 512), (700, 176), (2051, 512),
                                 (70000, 16), (262200, 32)])
def test_quantize(M, K):
    x = f32(rows(M, K, M + K))
    X = bf16(extremes(x, M) if K % 128 == 0 else x)
    a = A.fp8_quantize(dev(X))
    torch.cuda.synchronize()
    check_acts(a, f32(X).astype(np.float64), 0.0, (M, K))


@pytest.mark.parametrize("M,K", [(1, 16), (2, 28672), (37, 1072), (300, 512)])
def test_gated_quantize(M, K):
    X, g = rows(M, K, 5), rows(M, K, 6, gain=20.0)
    a = A.fp8_quantize(dev(X), gate=dev(g))
    torch.cuda.synchronize()
    p = gated(f32(X).astype(np.float64), f32(g).astype(np.float64))
    # exp and its argument (|g| 2^-24 absolute, at most 2 steps beside), 1 + e, division, two products: at most 7 half
    # steps, plus |g| of them from exp's argument
    check_acts(a, p, (7 + 2 * float(np.abs(f32(g)).max())) * H32, (M, K))


def test_gate_at_its_ends():
    g = np.tile(np.array([0.0, -0.0, 100.0, -100.0, 300.0, -300.0, 1e-30, -1e-30], np.float32), 16)
    a = A.fp8_quantize(dev(bf16(np.full((1, 128), 3, np.float32))), gate=dev(bf16(g[None])))
    v = O.code_value(u8(a.codes))[0, :8]
    assert np.array_equal(v, [0, 0, 144, 0, 448, 0, 0, 0])    # 900 -> 448, 300 -> 149.3
    for bad in (np.inf, -np.inf, np.nan):
        h = g.copy()
        h[3] = bad
        a = A.fp8_quantize(dev(bf16(np.ones((1, 128), np.float32))), gate=dev(bf16(h[None])))
        assert torch.isnan(a.scales).all() and not u8(a.codes).any()


@pytest.mark.parametrize("K,N", [(16, 1), (16, 64), (144, 70), (128, 128), (128, 300), (512, 257), (1024, 96), (4096, 8),
                                 (272, 1000)])
def test_pack(K, N):
    W = np.random.default_rng(K + N).standard_normal((K, N), dtype=np.float32) / np.sqrt(np.float32(K))
    W *= np.exp(np.linspace(-8, 8, N, dtype=np.float32))[None]
    if K > 1000:
        W[130, :] = 0
        W[:128] = 0
        W[300, 3] = np.nan
    W = bf16(W)
    q = A.fp8_pack(dev(W))
    torch.cuda.synchronize()
    packed = u8(q.codes)
    codes, s = O.weights_codes(packed, K, N), q.scales.cpu().numpy()
    assert np.array_equal(O.weights_layout(codes), packed)     # zeros past K and N
    w = f32(W).astype(np.float64)
    check_groups(codes, s, O.scale_of, w, 0.0, lambda v: O.spread_weights(v, K, N), O.weight_top(w), (K, N))


def test_pack_of_weights_at_any_address_and_what_lies_behind():
    K, N = 272, 200
    base = torch.from_numpy(np.random.default_rng(1).standard_normal(K * N + 8).astype(np.float32)).to(DEV, torch.bfloat16)
    W = base[1:1 + K * N].view(K, N)
    nc, ns = A.awq_fp8_codes_bytes(K, N), A.awq_fp8_scales_count(K, N)
    codes = torch.full((nc + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((ns + 64,), 7.0, device=DEV)
    A.awq_fp8_pack(W, codes[:nc].view(4, 3, 8, 64, 16), scales[:ns].view(2, 3))
    ref = A.fp8_pack(W.clone())
    torch.cuda.synchronize()
    assert torch.equal(codes[:nc], ref.codes.view(torch.uint8).flatten()) and torch.equal(scales[:ns], ref.scales.flatten())
    assert (codes[nc:] == 0x5A).all() and (scales[ns:] == 7).all()


def test_quantize_keeps_what_lies_behind_and_takes_any_address():
    M, K = 5, 144
    X = dev(rows(M, K, 2))
    codes = torch.full((M * K + 64,), 0x5A, dtype=torch.uint8, device=DEV)
    scales = torch.full((M * 2 + 9,), 7.0, device=DEV)
    A.awq_fp8_quantize(X, None, codes[:M * K].view(M, K).view(F8), scales[1:1 + 2 * M].view(M, 2))
    ref = A.fp8_quantize(X)
    torch.cuda.synchronize()
    assert torch.equal(codes[:M * K], ref.codes.view(torch.uint8).flatten()) and torch.equal(scales[1:1 + 2 * M], ref.scales.flatten())
    assert (codes[M * K:] == 0x5A).all() and scales[0] == 7 and (scales[1 + 2 * M:] == 7).all()
