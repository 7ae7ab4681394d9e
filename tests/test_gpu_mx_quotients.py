"""Division by the input scales at the ends of their range, on the GPU, against float64: quotients that
overflow, that fall below the smallest normal float32, that lie next to the border of two codes, and
norm weights whose quotient by a scale overflows although the result does not."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as O
from tests.mx_util import A, DEV, EPS32, act_buffers, bf16, check_quantized, dev, f32, host_acts

pytestmark = pytest.mark.gpu


def quotient(v: np.ndarray, s: np.ndarray) -> np.ndarray:
    """v / s rounded to float32 once.  Both have at most 24 significant bits, so the float64 quotient
    (53 >= 2 * 24 + 2) rounds to the same float32 as the exact one."""
    with np.errstate(all="ignore"):
        return (v.astype(np.float64) / s.astype(np.float64)).astype(np.float32)


SCALES = [2.0 ** -120, 1.9 * 2.0 ** -120, 2.0 ** -60 * 1.1, 0.64, 0.9999999, 1.0, 1.37, 3.1, 2.0 ** 24 * 1.7, 2.0 ** 120]


@pytest.mark.parametrize("scaled", [False, True])
def test_unpack_of_every_code_under_every_scale(scaled):
    """All sixteen codes under all 256 scale bytes, divided by scales over their whole range: the float32
    quotient rounded to bf16, infinities where it overflows, NaN for E = 255 alone."""
    N, K = 256, 32 * len(SCALES)
    c = np.tile(np.arange(16, dtype=np.uint8), K // 16)[:, None].repeat(N, 1)
    E = np.arange(N, dtype=np.uint8)[None].repeat(K // 32, 0)
    s = np.repeat(np.array(SCALES, np.float32), 32) if scaled else np.ones(K, np.float32)
    codes, scales = (torch.from_numpy(a).to(DEV) for a in O.weights_layout(c, E))
    W = torch.full((K, N), 7.0, dtype=torch.bfloat16, device=DEV)
    A.awq_mx_unpack(codes, scales, torch.from_numpy(s).to(DEV) if scaled else None, W)
    v = O.values(c.T.copy(), E.T.copy(), 4).T               # float64: no value is rounded
    with np.errstate(all="ignore"):
        q = (v / s.astype(np.float64)[:, None]).astype(np.float32)
    want = torch.from_numpy(q).to(torch.bfloat16).float().numpy()
    got = f32(W)
    assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:4]
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(got != want)[:4]
    assert np.isinf(want).any() and (np.isnan(want) == (E == 255).repeat(32, 0)).all()


def test_pack_and_back_where_the_way_back_overflows():
    """Weights near the largest bf16 times 0.65, 5.04 times 2^125, round up to element 6; divided again
    they pass the largest number and are infinite, not NaN."""
    K, N = 32, 8
    W = bf16(np.where(np.arange(K * N).reshape(K, N) % 2, 3.3e38, -3.3e38))
    s = np.full(K, 0.65, np.float32)
    codes, scales = O.pack(f32(W), s)
    assert scales[0, 0, 0] == 252 and set(O.unpair(codes[0, 0, :N]).ravel()) == {7, 15}
    back = f32(A.mx_unpack(A.mx_pack(dev(W), torch.from_numpy(s).to(DEV))))
    assert np.array_equal(back, np.where(f32(W) > 0, np.inf, -np.inf))


def border_columns(tiny: bool, seed: int, bits: int):
    """(p bf16 [R, K], s float32 [K]): most quotients p / s lie within two float32 steps of the border of
    two codes under their block's scale, which the block's first channel sets."""
    rng = np.random.default_rng(seed)
    R, K = 1, 4096
    top = 6.0 if bits == 4 else 448.0
    t = O.MAGNITUDES[bits]
    border = (t[2:] + t[1:-1]) / 2
    e = rng.integers(-124, -95, K // 32) if tiny else rng.integers(-20, 20, K // 32)
    E = np.repeat(2.0 ** e.astype(np.float64), 32)
    mantissa = 1 + rng.integers(0, 128, K) / 128
    at = rng.choice(border, K) * E
    # p within a factor of two of the border, so that s lies near 1
    p = mantissa * 2.0 ** np.floor(np.log2(at)) * rng.choice([-1.0, 1.0], K)
    s = (np.abs(p) / at).astype(np.float32)
    s = (s.view(np.int32) + rng.integers(-1, 2, K)).astype(np.int32).view(np.float32)
    p[::32], s[::32] = (top * E)[::32], 1.0
    return bf16(p[None].astype(np.float32)), s


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("tiny", [False, True])
def test_quantize_next_to_borders(bits, tiny):
    for seed in range(4):
        X, s = border_columns(tiny, seed, bits)
        a = A.mx_quantize(dev(X), torch.from_numpy(s).to(DEV), bits)
        c, E, _ = host_acts(a.codes, a.scales)
        wc, wE = O.quantize(quotient(f32(X), s).astype(np.float64), bits)
        assert np.array_equal(E, wE)
        assert np.array_equal(c & (127 if bits == 8 else 7), wc & (127 if bits == 8 else 7)), \
            int((c != wc).sum())


def norm_of_ones(w: torch.Tensor, s: np.ndarray, bits: int):
    """The norm's codes of a row of +-1 (root mean square 1, eps below every rounding): y = +-w exactly."""
    K = w.numel()
    X = bf16(np.where(np.arange(K) % 3 == 0, -1.0, 1.0)[None])
    codes, scales = act_buffers(1, K, bits)
    A.awq_rms_norm(dev(X), None, dev(w), 1e-30, None, None, torch.from_numpy(s).to(DEV), codes, scales)
    return f32(X) * f32(w)[None], host_acts(codes, scales)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("tiny", [False, True])
@pytest.mark.parametrize("K", [512, 4096, 8192, 16384, 32768, 36864])
def test_norm_codes_next_to_borders(K, bits, tiny):
    """y / s is the float32 quotient that the quantizer forms, in every kernel of the norm."""
    p, s = (np.concatenate(v, -1) for v in zip(*[(f32(a), b) for a, b in (border_columns(tiny, i, bits) for i in range(9))]))
    w, s = bf16(p[0, :K]), s[:K].copy()
    y, (c, E, _) = norm_of_ones(w, s, bits)
    wc, wE = O.quantize(quotient(y, s).astype(np.float64), bits)
    assert np.array_equal(E, wE)
    assert np.array_equal(c & (127 if bits == 8 else 7), wc & (127 if bits == 8 else 7)), int((c != wc).sum())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K", [(3, 256), (3, 4096), (300, 8192), (2, 16384), (2, 40000)])
def test_norm_where_weight_over_scale_overflows(M, K, bits):
    """|w| / s beyond float32 in every channel, y / s inside it: small rows beside one large element, and zeros."""
    X = np.full((M, K), 2.0 ** -12)
    X[:, 0] = 2.0 ** 14
    X[1] = 0
    X[:, 64:128] = 0
    w, s = bf16(np.where(np.arange(K) == 0, 2.0 ** -40, 256.0)), np.full(K, 2.0 ** -120, np.float32)
    codes, scales = act_buffers(M, K, bits)
    A.awq_rms_norm(dev(bf16(X)), None, dev(w), 1e-5, None, None, torch.from_numpy(s).to(DEV), codes, scales)
    y = O.rms_norm(X, None, f32(w).astype(np.float64), 1e-5) / s
    assert np.abs(y).max() < 2.0 ** 127
    c, E, _ = host_acts(codes, scales)
    assert (E < 255).all(), int((E == 255).sum())
    assert not E[1].any() and not c[1].any() and not E[:, 2:4].any()
    check_quantized(codes, scales, y, 8 * EPS32, (M, K, bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** 120])
def test_norm_at_the_ends_of_the_scales(scale, bits):
    """The smallest and largest scales with weights to either side: the float32 quotient, subnormal or
    infinite where it is."""
    K = 512
    rng = np.random.default_rng(1)
    w = (1 + rng.integers(0, 128, K) / 128) * 2.0 ** np.repeat(rng.integers(-16, 12, K // 32), 32)
    y, (c, E, _) = norm_of_ones(bf16(w), np.full(K, scale, np.float32), bits)
    q = quotient(y, np.full(K, scale, np.float32)).astype(np.float64)
    wc, wE = O.quantize(q, bits)
    assert np.array_equal(E, wE) and (scale > 1 or (wE == 255).any())
    assert np.array_equal(c & (127 if bits == 8 else 7), wc & (127 if bits == 8 else 7))


@pytest.mark.parametrize("bits", [8, 4])
def test_subnormal_numbers(bits):
    """Numbers down to the smallest bf16 (2^-133), in the quantizer, the packing and back."""
    rng = np.random.default_rng(3)
    u = (rng.integers(0, 2 ** 9, (64, 256)) | (rng.integers(0, 2, (64, 256)) << 15)).astype(np.uint16)
    X = torch.from_numpy(u.view(np.int16).copy()).view(torch.bfloat16)
    mask = 127 if bits == 8 else 7
    a = A.mx_quantize(dev(X), bits=bits)
    c, E, _ = host_acts(a.codes, a.scales)
    wc, wE = O.quantize(f32(X).astype(np.float64), bits)
    assert np.array_equal(E, wE) and np.array_equal(c & mask, wc & mask)
    if bits == 4:
        for s in (None, np.full(64, 1.0, np.float32)):
            q = A.mx_pack(dev(X), None if s is None else torch.from_numpy(s).to(DEV))
            codes, scales = O.pack(f32(X), s)
            assert np.array_equal(q.scales.view(torch.uint8).cpu().numpy(), scales)
            assert np.array_equal(O.unpair(q.codes.cpu().numpy()) & 7, O.unpair(codes) & 7)
            want = torch.from_numpy(O.weights_values(codes, scales, 64, 256).astype(np.float32)).to(torch.bfloat16)
            assert np.array_equal(f32(A.mx_unpack(q)), f32(want))
