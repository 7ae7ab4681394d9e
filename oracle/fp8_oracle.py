"""Plain float64 oracle of the 8-bit operators (numpy; test infrastructure only): e4m3 groups of 128 with
float32 scales and their packed layout, and the 8-bit cache with its append and attention.
"""
from __future__ import annotations

import numpy as np

from .mx_oracle import code_values, round_codes

GROUP = 128
LEAST = 448.0 * 2.0 ** -120


# ---------------------------------------------------------------- groups of 128
def scale_of(top: np.ndarray) -> np.ndarray:
    """Largest magnitudes (float64 of float32 numbers) -> scales float32; NaN where one is not finite."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.maximum(np.where(np.isfinite(top), top, 0.0), LEAST).astype(np.float32) / np.float32(448)
    return np.where(np.isfinite(top), s, np.float32(np.nan)).astype(np.float32)


def group_top(p: np.ndarray) -> np.ndarray:
    """p float64 [R, K] -> the largest magnitude of each group [R, ceil(K/128)], infinite where one is not finite."""
    R, K = p.shape
    c = -(-K // GROUP)
    b = np.zeros((R, c * GROUP))
    b[:, :K] = np.where(np.isfinite(p), np.abs(p), np.inf)
    return b.reshape(R, c, GROUP).max(-1)


def weight_top(W: np.ndarray) -> np.ndarray:
    """W float64 [K, N] -> [ceil(N/128), ceil(K/128)]."""
    t = group_top(W.T)                                         # [N, Kc]
    nb = -(-t.shape[0] // GROUP)
    b = np.zeros((nb * GROUP, t.shape[1]))
    b[:t.shape[0]] = t
    return b.reshape(nb, GROUP, -1).max(1)


def spread_rows(s: np.ndarray, K: int) -> np.ndarray:
    return np.repeat(s.astype(np.float64), GROUP, axis=1)[:, :K]


def spread_weights(s: np.ndarray, K: int, N: int) -> np.ndarray:
    """[Nb, Kc] -> [K, N]."""
    return np.repeat(np.repeat(s.T.astype(np.float64), GROUP, 0)[:K], GROUP, 1)[:, :N]


def weights_layout(c: np.ndarray) -> np.ndarray:
    """codes [K, N] -> [Nt, Kc, 8, 64, 16], by the definition of every byte's place."""
    K, N = c.shape
    out = np.zeros((-(-N // 64), -(-K // GROUP), 8, 64, 16), np.uint8)
    k, n = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
    out[n // 64, k // 128, 2 * (n % 64 // 16) + k % 128 // 64, 16 * (k % 64 // 16) + n % 16, k % 16] = c
    return out


def weights_codes(packed: np.ndarray, K: int, N: int) -> np.ndarray:
    k, n = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
    return packed[n // 64, k // 128, 2 * (n % 64 // 16) + k % 128 // 64, 16 * (k % 64 // 16) + n % 16, k % 16]


# ---------------------------------------------------------------- cache
def cache_byte(top: float) -> int:
    """The least E >= 0 with top <= 448 * 2^(E - 127); 255 for what is not finite or would round to 2^128 under it."""
    if not top < 1.9375 * 2.0 ** 127:
        return 255
    E = 0
    if top > 0:
        E = max(int(np.floor(np.log2(top))) + 127 - 9, 0)
        while top > 448 * 2.0 ** (E - 127):
            E += 1
    return E


def v_rows(v: np.ndarray) -> np.ndarray:
    """V codes [blocks, Hk, T/16, D, 16] -> [blocks, Hk, T, D]."""
    b, h, t, d, _ = v.shape
    return v.transpose(0, 1, 2, 4, 3).reshape(b, h, t * 16, d)


def v_layout(v: np.ndarray) -> np.ndarray:
    b, h, t, d = v.shape
    return np.ascontiguousarray(v.reshape(b, h, t // 16, 16, d).transpose(0, 1, 2, 4, 3))


def head_norm(x: np.ndarray, weight, eps: float) -> np.ndarray:
    if weight is None:
        return x
    with np.errstate(invalid="ignore", over="ignore"):
        return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight


def rotate(x: np.ndarray, turn, R: int, interleaved: bool):
    """x [n, H, D], turn [n, R] -> (rotated, what its rounding errors are relative to)."""
    if turn is None:
        return x, np.abs(x)
    cos, sin = turn[:, None, :R // 2], turn[:, None, R // 2:]
    first = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
    second = first + (1 if interleaved else R // 2)
    y, size = x.copy(), np.abs(x)
    with np.errstate(invalid="ignore", over="ignore"):
        a, c = x[..., first], x[..., second]
        y[..., first], y[..., second] = a * cos - c * sin, c * cos + a * sin
        size[..., first] = np.abs(a * cos) + np.abs(c * sin)
        size[..., second] = np.abs(c * cos) + np.abs(a * sin)
    return y, size


def attention(q, k, v, causal: bool, scale: float):
    """One head of one sequence, float64: q [n, D] at the last n positions of k, v [L, D] (None where a token is
    missing: seen by nobody; a query at a position below zero sees none).  Returns (out, sum p |v| / sum p, the largest
    |q| . |k| * scale)."""
    n, D = q.shape
    L = k.shape[0]
    pos = np.arange(L - n, L)
    seen = np.arange(L)[None, :] <= (pos[:, None] if causal else L)
    seen = seen & ~np.isnan(k).all(-1)[None, :] if np.isnan(k).any() else seen
    out, size = np.zeros((n, D)), np.zeros((n, D))
    kk = np.nan_to_num(k, nan=0.0)
    vv = np.nan_to_num(v, nan=0.0)
    s = np.where(seen, q @ kk.T * scale, -np.inf)
    any_ = seen.any(1) & (pos >= 0)
    m = np.where(any_, s.max(1, initial=-np.inf), 0.0)
    p = np.where(any_[:, None], np.exp(s - m[:, None]), 0.0)
    total = np.where(any_, p.sum(1), 1.0)
    out, size = p @ vv / total[:, None], p @ np.abs(vv) / total[:, None]
    reach = float((np.abs(q) @ np.abs(kk).T).max(initial=0.0)) * abs(scale)
    return out, size, reach


def codes_of(x: np.ndarray) -> np.ndarray:
    return round_codes(x, 8)


def code_value(c: np.ndarray) -> np.ndarray:
    return code_values(c, 8)
