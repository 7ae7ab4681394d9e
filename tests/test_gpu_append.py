"""q|k|v normed, rotated and appended to the 8-bit cache, on the GPU against float64: q, every slot and scale byte of the cache,
blocks begun and joined, slots and blocks that nothing reaches, tokens and blocks that fit nothing."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.fp8_util import A, DEV, H32, HBF, Batch, bf16, dev, f32

pytestmark = pytest.mark.gpu
EPS = 1e-5


def rope_table(P, R):
    a = np.arange(P)[:, None] * 10000.0 ** (-np.arange(R // 2) * 2 / R)
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def inputs(B, R, norm, P=None, sizes=None, seed=1):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B.M, B.Hq + 2 * B.Hk, B.D)).astype(np.float32)
    if sizes is not None:
        x *= sizes.astype(np.float32)[:, None, None]
    w = [bf16(1 + 0.2 * rng.standard_normal(B.D)) if norm else None for _ in range(2)]
    P = max(max(L for L, _ in B.lengths), 1) if P is None else P
    return dict(qkv=bf16(x.reshape(B.M, -1)), qw=w[0], kw=w[1], rope=rope_table(P, R) if R else None)


def append(B, x, interleaved=False, max_q=None):
    d = B.d
    q = torch.full((B.M, B.Hq, B.D), 7.0, dtype=torch.bfloat16, device=DEV)
    A.awq_qkv_append(dev(x["qkv"]), dev(x["qw"]), dev(x["kw"]), EPS,
                     None if x["rope"] is None else torch.from_numpy(x["rope"]).to(DEV), interleaved, d["cu"], d["length"],
                     d["table"], B.max_q if max_q is None else max_q, q, d["k"], d["v"], d["E"])
    torch.cuda.synchronize()
    return f32(q).astype(np.float64)


def check(B, x, q, interleaved=False, label=""):
    """Everything that the append may have written against its definition, everything else against what was there."""
    T, D, Hq, Hk = B.T, B.D, B.Hq, B.Hk
    rope = x["rope"]
    R, P = (0, 1 << 40) if rope is None else (rope.shape[1], rope.shape[0])
    rows = f32(x["qkv"]).astype(np.float64).reshape(B.M, Hq + 2 * Hk, D)
    wt = [None if x[n] is None else f32(x[n]).astype(np.float64) for n in ("qw", "kw")]
    k1, v1, E1 = B.download()
    k0, v0, E0 = B.k.copy(), B.v.copy(), B.E.copy()
    mine = np.zeros(B.M, bool)
    for b, (L, n) in enumerate(B.lengths):
        mine[B.cu[b]:B.cu[b] + n] = True
        pos = np.arange(L - n, L)
        r = np.arange(B.cu[b], B.cu[b] + n)
        ok = (pos >= 0) & (pos < P)
        assert not q[r[~ok]].any(), (label, b, "q of tokens without a position")
        pos, r = pos[ok], r[ok]
        if not len(r):
            continue
        turn = None if rope is None else rope[pos].astype(np.float64)
        # norm: the factor's rounding, two products; rotation: cosine, sine and sum: at most 6 half steps of |a cos| + |c sin|
        hq, sq = O.rotate(O.head_norm(rows[r, :Hq], wt[0], EPS), turn, R, interleaved)
        hk, sk = O.rotate(O.head_norm(rows[r, Hq:Hq + Hk], wt[1], EPS), turn, R, interleaved)
        err = np.abs(q[r] - hq)
        assert (err <= HBF * np.abs(hq) + 8 * H32 * sq + 1e-38).all(), (label, b, "q", err.max())
        for j in range(pos[0] // T, pos[-1] // T + 1):
            t = (pos // T) == j
            blk = B.table[b, j] if j < B.table.shape[1] else -1
            if not 0 <= blk < B.blocks:
                continue
            slots = pos[t] % T
            for i, (new, size, c0, c1) in enumerate(((hk, sk, k0, k1), (rows[r, Hq + Hk:], None, v0, v1))):
                for h in range(Hk):
                    p = new[t][:, h]
                    e = 8 * H32 * size[t][:, h] + 1e-38 if size is not None else np.zeros_like(p)
                    old = int(E0[blk, h, i]) if slots[0] else 0
                    top = np.abs(p)
                    lo, hi = (max(O.cache_byte(float(np.max(v))), old) for v in (np.maximum(top - e, 0), top + e))
                    got = int(E1[blk, h, i])
                    assert lo <= got <= hi, (label, b, j, h, i, lo, got, hi)
                    if got == 255:
                        assert not (c1[blk, h, slots] & 127).any()
                        want_old = c0[blk, h, :slots[0]]
                    else:
                        s = 2.0 ** (got - 127.0)
                        v = O.code_value(c1[blk, h, slots])
                        a, z = (O.code_value(O.codes_of(np.clip(u / s, -448, 448))) for u in (p - e, p + e))
                        assert ((v >= a) & (v <= z)).all(), (label, b, j, h, i)
                        want_old = c0[blk, h, :slots[0]]
                        if slots[0] and got > old:
                            want_old = O.codes_of(O.code_value(want_old) * 2.0 ** (old - got))
                    have = c1[blk, h, :slots[0]]
                    assert np.array_equal(np.where(have == 128, 0, have), np.where(want_old == 128, 0, want_old)), \
                        (label, b, j, h, i, "older tokens")
                    c0[blk, h, :slots[0]], c0[blk, h, slots], E0[blk, h, i] = have, c1[blk, h, slots], got
    assert np.array_equal(k0, k1) and np.array_equal(v0, v1) and np.array_equal(E0, E1), (label, "what nothing reaches")
    assert (q[~mine] == 7).all(), (label, "rows that no sequence has")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (8, 1), (6, 2)])
def test_sizes(D, T, Hq, Hk):
    for seed, (R, norm, il) in enumerate(((D, True, False), (D // 2, False, True), (0, True, False), (16, False, False))):
        lengths = [(1, 1), (T, T), (T + 1, 1), (2 * T + 5, 3), (3 * T + 7, 2 * T + 9), (5, 5), (T - 1, 2), (40, 0)]
        B = Batch(lengths, Hq, Hk, D, T, seed)
        B.upload()
        x = inputs(B, R, norm, seed=seed)
        check(B, x, append(B, x, il), il, (D, T, Hq, Hk, R, norm, il))


def test_growing_scales_token_by_token():
    """One sequence, token by token, each larger than the last: every step rescales what the block holds."""
    Hq, Hk, D, T = 4, 2, 64, 32
    for step in range(1, 40):
        if step == 1:
            B = Batch([(1, 1)], Hq, Hk, D, T, 3)
            B.table = np.array([[1, 0, 2]], np.int32)
            state = None
        B.lengths = [(step, 1)]
        if state is not None:
            B.k, B.v, B.E = state
        B.upload()
        x = inputs(B, 64, False, sizes=np.full(B.M, 1.6 ** (step % 23) * 0.01), seed=step)
        check(B, x, append(B, x), label=step)
        state = tuple(a.copy() for a in B.download())


def test_scale_jumps_beyond_all_codes():
    """A token 2^40 and 2^200 times larger than the block's older ones: those become zero."""
    for big in (2.0 ** 40, 2.0 ** 100, 3e38):
        B = Batch([(10, 1)], 2, 1, 128, 16, 5)
        B.E[:] = 60 if big > 2.0 ** 50 else 110
        B.upload()
        x = inputs(B, 0, False, sizes=np.full(B.M, 1.0))
        v = f32(x["qkv"])
        v[0, 3 * 128 - 1], v[0, 4 * 128 - 1] = big, -big
        x["qkv"] = bf16(v)
        check(B, x, append(B, x), label=big)


def test_infinities_and_nan_mark_the_block_of_their_head():
    for bad in (np.inf, -np.inf, np.nan):
        for first in (0, 7):
            B = Batch([(first + 3, 3)], 4, 2, 64, 16, 6)
            B.upload()
            x = inputs(B, 0, False)
            v = f32(x["qkv"]).reshape(B.M, 8, 64)
            v[1, 4, 9], v[2, 7, 11] = bad, bad              # K of head 0, V of head 1
            x["qkv"] = bf16(v.reshape(B.M, -1))
            q = append(B, x)
            _, _, E = B.download()
            blk = B.table[0, 0]
            assert E[blk, 0, 0] == 255 and E[blk, 1, 1] == 255 and E[blk, 1, 0] < 255 and E[blk, 0, 1] < 255
            check(B, x, q, label=(bad, first))
            # and it stays marked
            B.k, B.v, B.E = (a.copy() for a in B.download())
            B.lengths = [(first + 5, 2)]
            B.cu = np.array([0, 2], np.int32)
            B.upload()
            x = inputs(B, 0, False, seed=9)
            check(B, x, append(B, x), label="later")


def test_zeros_subnormals_and_norm_of_extremes():
    B = Batch([(6, 6), (4, 1)], 2, 1, 128, 16, 7)
    B.upload()
    x = inputs(B, 128, True)
    v = f32(x["qkv"])
    v[0] = 0
    v[1] = 1e-39
    v[2] = 3e38
    v[3, ::2] = 0
    x["qkv"] = bf16(v)
    check(B, x, append(B, x), label="extremes")


def test_tokens_and_blocks_that_fit_nothing():
    """Lengths below the new tokens, blocks outside the cache or the table, positions past the rotation's table, rows past
    max_q: nothing of it faults, and what is there is written."""
    Hq, Hk, D, T = 4, 2, 64, 16
    B = Batch([(70, 70), (20, 20), (50, 3), (33, 33)], Hq, Hk, D, T, 8, lead=2)
    B.table[0, 1], B.table[0, 3] = -1, B.blocks
    B.table = B.table[:, :4].copy()                         # sequence 0 reaches past the table
    B.table[2, 3] = np.iinfo(np.int32).min
    B.lengths[1] = (7, 20)                                  # 13 tokens at negative positions
    B.lengths[3] = (-5, 33)                                 # none has a position
    B.upload()
    x = inputs(B, 64, True, P=60)                           # positions 60 .. 69 have no rotation
    check(B, x, append(B, x), label="fits nothing")
    # rows past max_q are left out
    B = Batch([(40, 40), (9, 9)], Hq, Hk, D, T, 9)
    B.upload()
    x = inputs(B, 64, True)
    q = append(B, x, max_q=9)
    assert (q[9:40] == 7).all() and not (q[:9] == 7).any() and not (q[40:49] == 7).any()


def test_cu_that_decreases_or_leaves_the_rows():
    """Bounds of a cu are the one before it and the rows; of the third sequence's rows 3 .. M - 1 max_q = 7 are taken."""
    B = Batch([(5, 5), (6, 6), (7, 7)], 2, 1, 64, 16, 10)
    B.cu = np.array([-4, 5, 3, 1000], np.int32)             # sequence 0: rows 0 .. 4; 1: none; 2: rows 3 .. M - 1
    B.upload()
    x = inputs(B, 0, False)
    q = append(B, x)
    left = (q == 7).all(axis=(1, 2))
    assert B.max_q == 7 and not left[:10].any() and left[10:].all()


def test_last_rows_and_blocks_of_many_sequences():
    B = Batch([(int(n), int(min(n, 1 + n % 5))) for n in np.random.default_rng(0).integers(1, 150, 130)], 3, 3, 64, 32, 11)
    B.upload()
    x = inputs(B, 32, True)
    check(B, x, append(B, x), label="many")
