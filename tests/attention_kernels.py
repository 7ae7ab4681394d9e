"""Calls that take a given kernel of the attention whatever their sequences hold: the plan goes by max_q and by the table's width,
and both may be larger than the sequences need.  tests/test_attention_kernels_plan.py holds this to the plan."""
import numpy as np

from oracle import fp8_oracle as O
from tests.fp8_util import attention_bound, f32

HEADS = [(16, 1), (32, 2)]                              # (heads of q, of the cache)
MOST_SEQUENCES = 3
# rows a workgroup: (max_q, tokens that the table covers); 16: as the sequences are, a few rows
WIDE = {128: (100, 4096), 256: (1300, 16384)}


def take(B, rows):
    """Makes batch B (tests/fp8_util.py), not yet uploaded, a call of the kernel of 16, 128 or 256 rows."""
    assert (B.Hq, B.Hk) in HEADS and len(B.lengths) <= MOST_SEQUENCES
    if rows == 16:
        assert B.max_q * B.Hq // B.Hk <= 16
        return B
    max_q, tokens = WIDE[rows]
    assert B.max_q <= max_q and B.table.shape[1] * B.T <= tokens
    B.max_q, B.M = max_q, max(B.M, max_q)
    rest = np.full((len(B.lengths), tokens // B.T - B.table.shape[1]), -1, np.int32)
    B.table = np.concatenate((B.table, rest), 1)
    return B


def tile_bound(out, size, reach, D, L):
    """|error| allowed of the kernels that take p with eight bits in the second product and in the sum alike: 128 and 256 rows.
    With p' = p (1 + d), |d| <= u = 2^-8, the result is off by sum p d (v - out) / sum p', at most u / (1 - u) of sum p |v - out| /
    sum p, which is at most size + |out|.  tests/fp8_util.py's bound has u size of it: the rest is u (1 + 2 u) |out| and 2 u^2 size.
    (A row of 8 tokens whose v are .56 once and near zero else, by hand in float64: off by 1.5e-4 with out = .0322 and size = .0327,
    u size = 1.3e-4.)"""
    u = 2.0 ** -8
    return attention_bound(out, size, reach, D, L) + u * (1 + 2 * u) * np.abs(out) + 2 * u * u * size


def check(B, rows, q, got, causal=True, scale=None, label=""):
    """tests/fp8_util.py's check with the bound of the kernel."""
    scale = B.D ** -0.5 if scale is None else scale
    x, y, G = f32(q).astype(np.float64), f32(got).astype(np.float64), B.Hq // B.Hk
    bound = attention_bound if rows == 16 else tile_bound
    mine = np.zeros(B.M, bool)
    for b, (L, n) in enumerate(B.lengths):
        r = slice(B.cu[b], B.cu[b] + n)
        mine[r] = True
        k, v = B.cached(b)
        for h in range(B.Hq):
            out, size, reach = O.attention(x[r, h], k[:, h // G], v[:, h // G], causal, scale)
            ok = np.abs(y[r, h] - out) <= bound(out, size, reach, B.D, L)
            assert ok.all(), (label, b, h, np.argwhere(~ok)[:4].tolist(), y[r, h][~ok][:4], out[~ok][:4])
    assert (y[~mine] == 7).all(), (label, "rows that no sequence has")
