"""Inputs and bounds shared by the GPU tests of the 8-bit operators."""
import numpy as np
import torch

from oracle import fp8_oracle as O
from tests.mx_util import A, DEV, bf16, dev, f32, product_bound, rows  # noqa: F401

H32 = 2.0 ** -24      # half a step of float32, relative
HBF = 2.0 ** -8       # half a step of bf16, relative
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def u8(t: torch.Tensor) -> np.ndarray:
    return t.view(torch.uint8).cpu().numpy()


def values8(t: torch.Tensor) -> np.ndarray:
    return O.code_value(u8(t))


def between(codes: np.ndarray, lo: np.ndarray, hi: np.ndarray, label) -> None:
    """Codes stand for numbers between the roundings of lo and hi: rounding is monotone."""
    v, a, b = (O.code_value(codes), *(O.code_value(O.codes_of(x)) for x in (lo, hi)))
    bad = ~((v >= np.minimum(a, b)) & (v <= np.maximum(a, b)))
    assert not bad.any(), (label, np.argwhere(bad)[:4].tolist(), v[bad][:4], lo[bad][:4], hi[bad][:4])


def check_groups(codes: np.ndarray, s: np.ndarray, s_of, p: np.ndarray, delta: float, spread, top: np.ndarray, label):
    """codes, s are the quantization of numbers within p (1 +- delta) (float64): s is the scale of a largest
    magnitude within as much, and a code the rounding of the number over that s, up to two more units in the last place
    of float32 (2^-22).  spread(s): the scales at the numbers; top: the groups' largest magnitudes."""
    lo, hi = s_of(top * (1 - delta)), s_of(top * (1 + delta))
    nan = np.isnan(lo)
    assert np.array_equal(np.isnan(s), nan), (label, np.argwhere(np.isnan(s) != nan)[:4])
    assert ((s >= lo) & (s <= hi))[~nan].all(), (label, np.argwhere(~((s >= lo) & (s <= hi)) & ~nan)[:4])
    at = spread(s)
    bad = np.isnan(at)
    assert not (codes[bad] & 127).any(), label
    with np.errstate(invalid="ignore"):
        q = np.where(bad, 0.0, p / np.where(bad, 1.0, at))
    d = delta + 2.0 ** -22
    between(codes, q * (1 - d), q * (1 + d), label)


def random_acts(M, K, seed):
    """Random codes and scales of activations on the device, and their float64 values."""
    rng = np.random.default_rng(seed)
    c = (rng.integers(0, 127, (M, K)) | rng.integers(0, 2, (M, K)) * 128).astype(np.uint8)
    s = np.exp(rng.uniform(-9, 3, (M, -(-K // 128)))).astype(np.float32)
    return torch.from_numpy(c).to(DEV).view(F8), torch.from_numpy(s).to(DEV), O.code_value(c) * O.spread_rows(s, K)


def random_weights(K, N, seed):
    rng = np.random.default_rng(seed)
    c = (rng.integers(0, 127, (K, N)) | rng.integers(0, 2, (K, N)) * 128).astype(np.uint8)
    s = np.exp(rng.uniform(-9, 3, (-(-N // 128), -(-K // 128)))).astype(np.float32)
    return (torch.from_numpy(O.weights_layout(c)).to(DEV).view(F8), torch.from_numpy(s).to(DEV),
            O.code_value(c) * O.spread_weights(s, K, N))


def product(xc, xs, wc, ws_, N, ws=None):
    M, K = xc.shape
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    if ws is None:
        ws = A.workspace(A.awq_fp8_gemm_workspace_size(M, K, N), DEV)
    A.awq_fp8_gemm(xc, xs, wc, ws_, Y, ws)
    torch.cuda.synchronize()
    return Y


def check_product(Y, x, w, label):
    """Y against the float64 product of x [M, K] and w [K, N].  The bound is that of the other 8-bit product: half a step of
    the result, a float32 step of sum |x w| for each group's sum and join (here K/128 groups, each with a scale's product
    and an addition, under the K/32 + 64 steps counted there), and the matrix core's cuts, 2^-10 of sum |x w|."""
    x, w = (torch.from_numpy(v).to(Y.device) if isinstance(v, np.ndarray) else v for v in (x, w))
    y, got = x @ w, Y.double()
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan), (label, int(torch.isnan(got).sum()), int(nan.sum()))
    x, w, y = (torch.nan_to_num(v, nan=0.0) for v in (x, w, y))
    bad = ~nan & ~((got - y).abs() <= product_bound(x, w, y, 8))
    assert not bad.any(), (label, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), y[bad][:4].tolist())


# ---------------------------------------------------------------- cache
class Batch:
    """Sequences of given (tokens, new tokens) over a cache whose blocks lie in random order, filled with random
    codes (NaN codes among them where no token of any sequence lies) and scales."""

    def __init__(self, lengths, Hq, Hk, D, T, seed=0, spare=2, lead=0):
        rng = np.random.default_rng(seed)
        self.lengths, self.Hq, self.Hk, self.D, self.T = lengths, Hq, Hk, D, T
        used = [-(-L // T) for L, _ in lengths]
        self.blocks = sum(used) + spare
        order = rng.permutation(self.blocks).astype(np.int32)
        self.table = np.full((len(lengths), max(max(used), 1)), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.cu = (lead + np.concatenate(([0], np.cumsum([n for _, n in lengths])))).astype(np.int32)
        self.M, self.max_q = int(self.cu[-1]) + 3, max(max(n for _, n in lengths), 1)
        shape = (self.blocks, Hk, T, D)
        self.k, self.v = (rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2))
        self.E = rng.integers(115, 121, (self.blocks, Hk, 2)).astype(np.uint8)
        for b, (L, _) in enumerate(lengths):       # finite where tokens are
            for j in range(used[b]):
                n, blk = min(L - j * T, T), self.table[b, j]
                for c in (self.k, self.v):
                    t = c[blk, :, :n]
                    t[(t & 127) == 127] = 0x40
        self.rng = rng

    def upload(self):
        t = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
        self.d = dict(cu=t(self.cu), length=t(np.array([L for L, _ in self.lengths], np.int32)), table=t(self.table),
                      k=t(self.k.copy()).view(F8), v=t(O.v_layout(self.v)).view(F8), E=t(self.E.copy()))
        return self.d

    def download(self):
        return u8(self.d["k"]), O.v_rows(u8(self.d["v"])), u8(self.d["E"])

    def queries(self, scale=1.0):
        return bf16(self.rng.standard_normal((self.M, self.Hq, self.D)).astype(np.float32) * np.float32(scale))

    def cached(self, b):
        """K and V of sequence b [L, Hk, D], float64; NaN rows where its block is missing or marked."""
        L, T = self.lengths[b][0], self.T
        k, v = np.full((L, self.Hk, self.D), np.nan), np.full((L, self.Hk, self.D), np.nan)
        for j in range(-(-L // T)):
            blk = self.table[b, j] if j < self.table.shape[1] else -1
            n = min(L - j * T, T)
            if 0 <= blk < self.blocks:
                for out, c, i in ((k, self.k, 0), (v, self.v, 1)):
                    t = c[blk, :, :n]
                    x = O.code_value(np.where((t & 127) == 127, 0, t)) * 2.0 ** (self.E[blk, :, i].astype(float) - 127)[:, None, None]
                    out[j * T:j * T + n] = x.transpose(1, 0, 2)
        return k, v


def attend(B: Batch, q, causal=True, scale=None, ws=None, max_q=None):
    d = B.d
    out = torch.full((B.M, B.Hq, B.D), 7.0, dtype=torch.bfloat16, device=DEV)
    max_q = B.max_q if max_q is None else max_q
    if ws is None:
        ws = A.workspace(A.awq_attention_workspace_size(B.M, len(B.lengths), max_q, B.Hq, B.Hk, B.D), DEV)
    A.awq_attention(q, d["cu"], d["length"], d["table"], max_q, d["k"], d["v"], d["E"],
                    B.D ** -0.5 if scale is None else scale, causal, out, ws)
    torch.cuda.synchronize()
    return out


def attention_bound(out, size, reach, D, L):
    """|error| allowed.  size = sum p |v| / sum p, reach = the largest scale |q| . |k|.
    Exponent: a score is D products added in float32 (a step 2^-23 of `reach` each, as for truncation), times scale and log2 e
    (three half steps), less the maximum (one): (2 D + 4) half steps of reach, which is the relative error of p, with
    exp2's own step; it enters sum p v and sum p.  p is rounded to bf16 for the second product.  Sums of L terms, a half
    step each, and 64 joins and rescalings, in sum p v and sum p.  The result: half a step of bf16."""
    p = (2 * D + 4) * H32 * reach + 2 * H32
    return HBF * np.abs(out) + size * (HBF + 2 * p + 2 * (L + 64) * H32) + 2.0 ** -126


def check_attention(B: Batch, q, got, causal=True, scale=None, label=""):
    scale = B.D ** -0.5 if scale is None else scale
    x, y, G = f32(q).astype(np.float64), f32(got).astype(np.float64), B.Hq // B.Hk
    mine = np.zeros(B.M, bool)
    for b, (L, n) in enumerate(B.lengths):
        r = slice(B.cu[b], B.cu[b] + n)
        mine[r] = True
        k, v = B.cached(b)
        for h in range(B.Hq):
            out, size, reach = O.attention(x[r, h], k[:, h // G], v[:, h // G], causal, scale)
            ok = np.abs(y[r, h] - out) <= attention_bound(out, size, reach, B.D, L)
            assert ok.all(), (label, b, h, np.argwhere(~ok)[:4].tolist(), y[r, h][~ok][:4], out[~ok][:4])
    assert (y[~mine] == 7).all(), (label, "rows that no sequence has")
