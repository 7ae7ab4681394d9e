"""Plain float64 oracle of the microscaled (MX) operators (numpy; test infrastructure only).

A block is 32 consecutive channels with one scale byte E (2^(E - 127)) and e4m3 or e2m1 elements;
E = max(biased exponent of max|p| - e_max, 0), elements are rounded to nearest even by looking the
scaled number up between the format's values, and a block with an infinity or a NaN has E = 255 and
zero elements.  Numbers p are float32 where the operator defines a float32 number.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
EMAX = {8: 8, 4: 2}


def _e4m3_values() -> np.ndarray:
    """Magnitudes of codes 0..126 (127 is NaN), ascending."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


MAGNITUDES = {8: _e4m3_values(), 4: np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])}


def round_codes(v: np.ndarray, bits: int) -> np.ndarray:
    """float64 -> sign-and-magnitude codes (uint8), nearest, ties to the even code, saturating."""
    t = MAGNITUDES[bits]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(t, a, side="left"), 1, len(t) - 1)
    lo = hi - 1
    dl, dh = a - t[lo], t[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c + np.where(np.signbit(v), 8 if bits == 4 else 128, 0)).astype(np.uint8)


def code_values(c: np.ndarray, bits: int) -> np.ndarray:
    n = 8 if bits == 4 else 128
    if bits == 8 and np.any((c & 127) == 127):
        raise ValueError("NaN code")
    return np.where(c >= n, -1.0, 1.0) * MAGNITUDES[bits][c % n]


def scale_values(E: np.ndarray) -> np.ndarray:
    return np.where(E == 255, np.nan, 2.0 ** (E.astype(np.float64) - 127))


def quantize(p: np.ndarray, bits: int):
    """float64 numbers [R, K] -> (codes uint8 [R, K], E uint8 [R, K/32])."""
    R, K = p.shape
    b = p.reshape(R, K // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    _, ex = np.frexp(top)                                   # top = f 2^ex, f in [0.5, 1)
    E = np.where(top > 0, np.maximum(ex - 1 + 127 - EMAX[bits], 0), 0)
    c = round_codes(b / (2.0 ** (E - 127.0))[..., None], bits)
    c = np.where(bad[..., None], 0, c).astype(np.uint8)
    return c.reshape(R, K), np.where(bad, 255, E).astype(np.uint8)


def values(c: np.ndarray, E: np.ndarray, bits: int) -> np.ndarray:
    """codes [R, K], E [R, K/32] -> float64 [R, K]; a block with E = 255 is NaN."""
    R, K = c.shape
    with np.errstate(invalid="ignore"):
        return (code_values(c, bits).reshape(R, -1, BLOCK) * scale_values(E)[..., None]).reshape(R, K)


def pair(c: np.ndarray) -> np.ndarray:
    """4-bit codes [R, K] -> bytes [R, K/2], even channel in the low half."""
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def unpair(b: np.ndarray) -> np.ndarray:
    out = np.empty(b.shape[:-1] + (2 * b.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = b & 15, b >> 4
    return out


def scale_position(c: int) -> int:
    """Byte of column c (< 64) among a tile's 64 scale bytes."""
    return 4 * (c % 16) + c // 16


def weights_layout(c: np.ndarray, E: np.ndarray):
    """codes [K, N], E [K/32, N] -> the packed layout (codes [Nt, Kb, 64, 16], scales [Nt, Kb, 64])."""
    K, N = c.shape
    nt, kb = -(-N // 64), -(-K // 128) * 4
    codes, scales = np.zeros((nt, kb, 64, 16), np.uint8), np.zeros((nt, kb, 64), np.uint8)
    by_column = pair(c.T.copy()).reshape(N, K // BLOCK, 16)
    n = np.arange(N)
    codes[n // 64, :K // BLOCK, n % 64] = by_column
    position = np.array([scale_position(v) for v in range(64)])
    scales[n // 64, :K // BLOCK, position[n % 64]] = E.T
    return codes, scales


def weights_values(codes: np.ndarray, scales: np.ndarray, K: int, N: int) -> np.ndarray:
    """The float64 weights [K, N] that a packed layout stands for."""
    W = np.empty((K, N))
    for n in range(N):
        c = unpair(codes[n // 64, :K // BLOCK, n % 64].reshape(1, -1))
        W[:, n] = values(c, scales[n // 64, :K // BLOCK, scale_position(n % 64)][None], 4)[0]
    return W


def pack(W32: np.ndarray, s):
    """W float32 [K, N] (bf16 values), s float32 [K] or None -> packed layout."""
    p = W32 if s is None else (W32 * s[:, None]).astype(np.float32)
    c, E = quantize(p.astype(np.float64).T, 4)
    return weights_layout(c.T, E.T)


def gated(x: np.ndarray, g: np.ndarray) -> np.ndarray:
    """x silu(g), float64."""
    with np.errstate(over="ignore", invalid="ignore"):
        return x * g / (1.0 + np.exp(-g))


def rms_norm(x: np.ndarray, r, weight: np.ndarray, eps: float) -> np.ndarray:
    h = x if r is None else x + r
    return h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * weight
