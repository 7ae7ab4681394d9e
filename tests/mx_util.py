"""Inputs and bounds shared by the GPU tests of the microscaled operators."""
import numpy as np
import torch

from oracle import mx_oracle as O
from weight_only_int4_act_amd import awq as A
from weight_only_int4_act_amd import inputs as I

DEV = "cuda:0"
EPS32 = 2.0 ** -24    # half a step of float32, relative


def bf16(a) -> torch.Tensor:
    return I.to_bf16(np.asarray(a, np.float32))


def f32(t: torch.Tensor) -> np.ndarray:
    return t.float().cpu().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def rows(M, K, seed, gain=50.0):
    """Activations with one channel in a hundred `gain` times larger (bf16, CPU)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K), dtype=np.float32)
    x[:, rng.random(K) < 0.01] *= np.float32(gain)
    return bf16(x)


def host_acts(codes: torch.Tensor, scales: torch.Tensor):
    """(codes [M, K], E, bits) as numpy bytes."""
    bits = 8 if codes.dtype == torch.float8_e4m3fn else 4
    c = codes.view(torch.uint8).cpu().numpy()
    return (c if bits == 8 else O.unpair(c)), scales.view(torch.uint8).cpu().numpy(), bits


def check_quantized(codes, scales, p, delta, label):
    """The codes stand for numbers between the quantizations of p (1 - delta) and p (1 + delta) (both in
    float64), where delta bounds the relative error of the float32 number that was quantized: the
    quantizer is monotone in each element for a fixed E, and E is monotone in the block's maximum."""
    c, E, bits = host_acts(codes, scales)
    lo, hi = O.quantize(p * (1 - delta), bits), O.quantize(p * (1 + delta), bits)
    assert np.all((E == lo[1]) | (E == hi[1])), (label, np.argwhere((E != lo[1]) & (E != hi[1]))[:4])
    ok = np.zeros(c.shape, bool)
    for side in (lo, hi):        # codes under the block scale of either side
        same = np.repeat(E == side[1], O.BLOCK, axis=1)
        step = np.repeat(np.where(E == 255, 1.0, 2.0 ** (np.minimum(E, 254) - 127.0)), O.BLOCK, axis=1)
        with np.errstate(invalid="ignore", over="ignore"):
            q = np.where(np.repeat(E == 255, O.BLOCK, axis=1), 0.0, p) / step
        a = O.code_values(O.round_codes(np.nan_to_num(q * (1 - delta)), bits), bits)
        b = O.code_values(O.round_codes(np.nan_to_num(q * (1 + delta)), bits), bits)
        v = O.code_values(c, bits)
        ok |= same & (v >= np.minimum(a, b)) & (v <= np.maximum(a, b))
    assert ok.all(), (label, np.argwhere(~ok)[:4])


def product_bound(x, w, y, bits):
    """|error| allowed of Y = x w (float64 values).  With S = sum |x w|:
    half a bf16 step of the result, 2^-8 |y|; one float32 step (2^-23, as for truncation) of S for each
    of the K/32 block sums and for the few joins after them; below the smallest normal float32, any
    result.  With e4m3 activations the matrix core adds products in groups of eight consecutive channels,
    each cut off 13 binary places below 2^e, e the largest sum of the two operands' exponents in the group
    (observed with single products: beside 256 a product of 2^-5 counts, one of 2^-6 does not, unless it
    lies in another group).  2^e is at most the largest product of the group, so eight cuts lose less than
    8 2^-13 of it, and all groups together less than 2^-10 S.  e2m1 products are multiples of 1/4 below
    2^6, so nothing of them is cut off."""
    S = x.abs() @ w.abs()
    return 2.0 ** -8 * y.abs() + ((x.shape[1] / 32 + 64) * 2.0 ** -23 + (2.0 ** -10 if bits == 8 else 0)) * S + 2.0 ** -126


def check_product(Y, x, w, bits, label):
    """Y against the product of the float64 values x [M, K] and w [K, N] (numpy), computed in float64."""
    x, w = torch.from_numpy(x).to(Y.device), torch.from_numpy(w).to(Y.device)
    y, got = x @ w, Y.double()
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan), (label, int(torch.isnan(got).sum()), int(nan.sum()))
    x, w, y = (torch.nan_to_num(v, nan=0.0) for v in (x, w, y))
    bad = ~nan & ~((got - y).abs() <= product_bound(x, w, y, bits))
    assert not bad.any(), (label, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), y[bad][:4].tolist())


def act_buffers(M, K, bits):
    codes = torch.full((M, K if bits == 8 else K // 2), 0x55, dtype=torch.uint8, device=DEV)
    return codes.view(torch.float8_e4m3fn) if bits == 8 else codes, torch.full((M, K // 32), 0x55, dtype=torch.uint8,
                                                                               device=DEV)


def random_acts(M, K, bits, seed, lo=110, hi=140):
    """Random codes and scale bytes on the device, and their float64 values."""
    rng = np.random.default_rng(seed)
    E = rng.integers(lo, hi, (M, K // 32)).astype(np.uint8)
    c = rng.integers(0, 127 if bits == 8 else 8, (M, K)).astype(np.uint8)
    c |= (rng.integers(0, 2, (M, K)) * (128 if bits == 8 else 8)).astype(np.uint8)
    t = torch.from_numpy(c if bits == 8 else O.pair(c))
    codes = t.view(torch.float8_e4m3fn) if bits == 8 else t
    return codes.to(DEV), torch.from_numpy(E).to(DEV), O.values(c, E, bits)


def random_weights(K, N, seed, lo=110, hi=140):
    rng = np.random.default_rng(seed)
    c, E = rng.integers(0, 16, (K, N)).astype(np.uint8), rng.integers(lo, hi, (K // 32, N)).astype(np.uint8)
    codes, scales = O.weights_layout(c, E)
    return torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), O.values(c.T.copy(), E.T.copy(), 4).T


def product(xc, xs, wc, wsc, M, K, N, ws=None):
    bits = 8 if xc.dtype == torch.float8_e4m3fn else 4
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    if ws is None:
        ws = A.workspace(A.awq_mx_gemm_workspace_size(M, K, N, bits), DEV)
    A.awq_mx_gemm(xc, xs, wc, wsc, Y, ws)
    torch.cuda.synchronize()
    return Y
