"""MX packing, unpacking, activation quantization and the root-mean-square norm on the GPU against the
float64 oracle: bit for bit where the operator defines the float32 number that is quantized, and
between the two neighbouring quantizations where float32 arithmetic precedes it."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as O
from tests.mx_util import A, DEV, EPS32, act_buffers, bf16, check_quantized, dev, f32, host_acts, rows
from weight_only_int4_act_amd import inputs as I

pytestmark = pytest.mark.gpu


def extremes(x: np.ndarray, seed) -> np.ndarray:
    """Plants blocks of zeros, negative zeros, subnormals, format borders, the largest numbers, one
    infinity, one NaN into a copy of x [R, K] (where there are that many blocks)."""
    x = x.copy()
    b = x.reshape(-1, 32)
    rng = np.random.default_rng(seed)
    plant = [np.zeros(32), np.full(32, -0.0), np.full(32, 2.0 ** -130), np.array([6, 7.96875, 5, 3.5, 2.5, 1.75, 1.25, .75,
             .25, 0, 8, -5, -2.5, -.25, 1, -1] * 2), np.full(32, 3.3e38), np.full(32, -2.0 ** 120),
             np.r_[np.inf, np.ones(31)], np.r_[np.ones(31), np.nan], np.r_[2.0 ** 100, np.full(31, 2.0 ** -100)],
             np.array([448, 464, 17, 19, 2.0 ** -9, 2.0 ** -10, 256, 255] * 4)]
    at = rng.permutation(b.shape[0])[:len(plant)]
    for i, r in enumerate(at):
        b[r] = plant[i]
    return x


@pytest.mark.parametrize("K,N", [(32, 1), (32, 64), (96, 70), (128, 300), (512, 257), (1024, 96), (4096, 8)])
@pytest.mark.parametrize("scaled", [False, True])
def test_pack_matches_the_oracle_bit_for_bit(K, N, scaled):
    rng = np.random.default_rng(K + N)
    W = rng.standard_normal((N, K), dtype=np.float32) / np.sqrt(np.float32(K))
    W = bf16(extremes(W, K + N).T.copy())
    s = I.scale_vector(K, seed=K) if scaled else None
    q = A.mx_pack(dev(W), None if s is None else torch.from_numpy(s).to(DEV))
    back = A.mx_unpack(q)
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        codes, scales = O.pack(f32(W), s)
    assert np.array_equal(q.scales.view(torch.uint8).cpu().numpy(), scales)
    got = q.codes.cpu().numpy()
    # a negative number that rounds to zero may carry either sign
    a, b = O.unpair(got), O.unpair(codes)
    assert np.array_equal(np.where(a == 8, 0, a), np.where(b == 8, 0, b))
    v = O.weights_values(codes, scales, K, N)
    ref = (v.astype(np.float32) / s[:, None] if scaled else v.astype(np.float32))
    ref = torch.from_numpy(ref.astype(np.float32)).to(torch.bfloat16).float().numpy()
    assert np.array_equal(f32(back), ref, equal_nan=True)


def test_pack_and_unpack_keep_what_lies_behind_them():
    K, N = 96, 70
    nc, ns = A.awq_mx_codes_bytes(K, N), A.awq_mx_scales_bytes(K, N)
    codes, scales = (torch.full((n + 256,), 0x5A, dtype=torch.uint8, device=DEV) for n in (nc, ns))
    back = torch.full((K * N + 128,), 7.0, dtype=torch.bfloat16, device=DEV)
    W = dev(rows(K, N, 3))
    c, s = codes[:nc].view(2, 4, 64, 16), scales[:ns].view(2, 4, 64)
    A.awq_mx_pack(W, None, c, s)
    A.awq_mx_unpack(c, s, None, back[:K * N].view(K, N))
    torch.cuda.synchronize()
    assert (codes[nc:] == 0x5A).all() and (scales[ns:] == 0x5A).all() and (back[K * N:] == 7).all()
    assert not c[:, 3].any() and not s[:, 3].any() and not c[1, :, 6:].any()
    assert not s.view(2, 4, 16, 4).transpose(2, 3).reshape(2, 4, 64)[1, :, 6:].any()


@pytest.mark.parametrize("M,K", [(1, 32), (1, 8192), (3, 96), (5, 2080), (16, 28672), (129, 512), (700, 160),
                                 (257, 5120), (2051, 512)])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("scaled", [False, True])
def test_quantize_matches_the_oracle_bit_for_bit(M, K, bits, scaled):
    X = bf16(extremes(f32(rows(M, K, M + K)), M))
    s = I.scale_vector(K, seed=K) if scaled else None
    a = A.mx_quantize(dev(X), None if s is None else torch.from_numpy(s).to(DEV), bits)
    torch.cuda.synchronize()
    with np.errstate(over="ignore", invalid="ignore"):
        p = (f32(X) if s is None else f32(X) / s).astype(np.float64)
    c, E = O.quantize(p, bits)
    gc, gE, _ = host_acts(a.codes, a.scales)
    assert np.array_equal(gE, E)
    zero = 8 if bits == 4 else 128
    assert np.array_equal(np.where(gc == zero, 0, gc), np.where(c == zero, 0, c))


@pytest.mark.parametrize("M,K", [(1, 32), (2, 28672), (37, 1056), (300, 512)])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("scaled", [False, True])
def test_gated_quantize(M, K, bits, scaled):
    X, g = rows(M, K, 5), rows(M, K, 6, gain=20.0)
    s = I.scale_vector(K, seed=K) if scaled else None
    a = A.mx_quantize(dev(X), None if s is None else torch.from_numpy(s).to(DEV), bits, gate=dev(g))
    torch.cuda.synchronize()
    p = O.gated(f32(X).astype(np.float64), f32(g).astype(np.float64))
    p = p if s is None else p / s
    # exp and its argument (|g| 2^-24 absolute, at most 2 steps beside), 1 + e, division, two products
    # and the division by s: at most 8 half steps, plus |g| of them from exp's argument
    check_quantized(a.codes, a.scales, p, (8 + 2 * float(np.abs(f32(g)).max())) * EPS32, (M, K, bits))


def test_gate_at_its_ends():
    g = np.array([0.0, -0.0, 100.0, -100.0, 300.0, -300.0, 1e-30, -1e-30] * 4, np.float32)
    X = np.ones((1, 32), np.float32) * 3
    a = A.mx_quantize(dev(bf16(X)), gate=dev(bf16(g[None])), bits=8)
    c, E, _ = host_acts(a.codes, a.scales)
    v = O.values(c, E, 8)[0]
    assert np.array_equal(v[:8], [0, 0, 288, 0, 896, 0, 0, 0])    # E = 128: 150 -> 144, 450 -> 448
    for bad in (np.inf, -np.inf, np.nan):
        h = g.copy()
        h[3] = bad
        a = A.mx_quantize(dev(bf16(X)), gate=dev(bf16(h[None])), bits=8)
        c, E, _ = host_acts(a.codes, a.scales)
        assert E[0, 0] == 255 and not c.any()


@pytest.mark.parametrize("M,K", [(1, 32), (1, 8192), (2, 96), (7, 5120), (333, 512), (3, 28672), (2, 33024), (600, 64),
                                 (5, 4064), (9, 16416), (300, 5120), (257, 8192), (300, 9088), (257, 16384)])
@pytest.mark.parametrize("bits,residual,scaled", [(8, True, False), (4, True, True), (8, False, True), (4, False, False)])
def test_rms_norm(M, K, bits, residual, scaled):
    eps = 1e-5
    X, w = rows(M, K, M + K), bf16(1 + 0.1 * np.random.default_rng(K).standard_normal(K))
    r = rows(M, K, M + K + 1) if residual else None
    if M > 1:
        X[1] = 0
        if residual:
            r[1] = 0
    s = I.scale_vector(K, seed=K) if scaled else None
    codes, scales = act_buffers(M, K, bits)
    ro = torch.empty((M, K), dtype=torch.bfloat16, device=DEV) if residual else None
    Y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    A.awq_rms_norm(dev(X), dev(r), dev(w), eps, ro, Y, None if s is None else torch.from_numpy(s).to(DEV), codes, scales)
    torch.cuda.synchronize()
    x64, r64 = f32(X).astype(np.float64), None if r is None else f32(r).astype(np.float64)
    y = O.rms_norm(x64, r64, f32(w).astype(np.float64), eps)
    # h (one rounding), 1/rms (one, and h's in the mean), two products, one division: 8 half steps
    delta = 8 * EPS32
    check_quantized(codes, scales, y if s is None else y / s, delta, (M, K, bits))
    lo, hi = (torch.from_numpy(y * (1 + d)).to(torch.float32).to(torch.bfloat16).float().numpy() for d in (-2 * delta, 2 * delta))
    got = f32(Y)
    assert np.all((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi)))
    if residual:
        ref = torch.from_numpy(f32(X) + f32(r)).to(torch.bfloat16)
        assert torch.equal(ro.cpu(), ref)


@pytest.mark.parametrize("M,K", [(3, 8), (4, 40), (2, 8200), (1, 40000)])
def test_rms_norm_without_codes(M, K):
    X, w = rows(M, K, K), bf16(np.linspace(0.5, 1.5, K))
    Y = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    A.awq_rms_norm(dev(X), None, dev(w), 1e-6, None, Y)
    y = O.rms_norm(f32(X).astype(np.float64), None, f32(w).astype(np.float64), 1e-6)
    assert np.all(np.abs(f32(Y) - y) <= np.abs(y) * (2.0 ** -8 + 16 * EPS32))


def test_rms_norm_outputs_do_not_depend_on_which_are_asked():
    M, K = 19, 1024
    X, r, w = dev(rows(M, K, 1)), dev(rows(M, K, 2)), dev(bf16(np.linspace(0.5, 1.5, K)))
    codes, scales = act_buffers(M, K, 8)
    ro, Y = torch.empty_like(X), torch.empty_like(X)
    A.awq_rms_norm(X, r, w, 1e-5, ro, Y, None, codes, scales)
    for keep in ("codes", "Y", "ro"):
        c2, s2 = act_buffers(M, K, 8)
        ro2, Y2 = torch.empty_like(X), torch.empty_like(X)
        A.awq_rms_norm(X, r, w, 1e-5, ro2 if keep != "codes" else None, Y2 if keep != "codes" else None, None,
                       c2 if keep != "Y" else None, s2 if keep != "Y" else None)
        if keep != "codes":
            assert torch.equal(ro, ro2) and torch.equal(Y, Y2)
        if keep != "Y":
            assert torch.equal(codes.view(torch.uint8), c2.view(torch.uint8)) and torch.equal(scales, s2)


@pytest.mark.parametrize("K", [512, 8192, 40032])
def test_rms_norm_in_place(K):
    M = 6
    X, r, w = rows(M, K, 1), rows(M, K, 2), bf16(np.linspace(0.5, 1.5, K))
    ro, Y = torch.empty_like(dev(X)), torch.empty_like(dev(X))
    A.awq_rms_norm(dev(X), dev(r), dev(w), 1e-5, ro, Y)
    for ro_at, y_at in (("r", "X"), ("X", "r"), ("r", None), (None, "X")):
        b = {"X": dev(X), "r": dev(r)}
        A.awq_rms_norm(b["X"], b["r"], dev(w), 1e-5, b.get(ro_at), b[y_at] if y_at else torch.empty_like(b["X"]))
        if ro_at:
            assert torch.equal(b[ro_at], ro)
        if y_at:
            assert torch.equal(b[y_at], Y)


def test_rms_norm_extreme_rows():
    K = 256
    w = bf16(np.ones(K))
    X = np.zeros((6, K), np.float32)
    X[0] = 3e38                      # squares beyond float32
    X[1, 0] = 1e-38
    X[2] = 2.0 ** -120
    X[3, 5] = np.inf
    X[4, 7] = np.nan
    X[5] = -1e30
    codes, scales = act_buffers(6, K, 8)
    Y = torch.empty((6, K), dtype=torch.bfloat16, device=DEV)
    A.awq_rms_norm(dev(bf16(X)), None, dev(w), 1e-5, None, Y, None, codes, scales)
    y = f32(Y)
    assert np.all(y[0] == 1) and np.all(y[5] == -1)
    x = f32(bf16(X)).astype(np.float64)
    with np.errstate(all="ignore"):
        ref = O.rms_norm(x, None, np.ones(K), 1e-5)
    for i in (1, 2):
        assert np.all(np.abs(y[i] - ref[i]) <= 2.0 ** -8 * np.abs(ref[i]) + 2.0 ** -126)
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    _, E, _ = host_acts(codes, scales)
    assert np.array_equal(E[3] == 255, np.arange(8) == 0) and np.all(E[4] == 255)


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 4 GiB: the last rows of a [M, K] matrix with M K 2 bytes above 2^32."""
    K = 8192
    M = 2 ** 32 // (2 * K) + 3
    X = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    tail = dev(rows(4, K, 9))
    X[-4:] = tail
    w = dev(bf16(np.ones(K)))
    codes, scales = act_buffers(M, K, 8)
    A.awq_mx_quantize(X, None, None, codes, scales)
    a = A.mx_quantize(tail)
    assert torch.equal(codes[-4:].view(torch.uint8), a.codes.view(torch.uint8))
    assert torch.equal(scales[-4:], a.scales.view(torch.uint8)) and not scales[:-4].any()
    A.awq_rms_norm(X, None, w, 1e-5, None, None, None, codes, scales)
    c2, s2 = act_buffers(4, K, 8)
    A.awq_rms_norm(tail, None, w, 1e-5, None, None, None, c2, s2)
    assert torch.equal(codes[-4:].view(torch.uint8), c2.view(torch.uint8)) and torch.equal(scales[-4:], s2)


@pytest.mark.parametrize("bits", [8, 4])
def test_more_rows_than_a_grid_has(bits):
    """A wavefront takes more than two rows where the grid's second dimension would not hold their number."""
    M, K = 65535 * 8 + 5, 32
    X = dev(rows(64, K, 1)).repeat(M // 64 + 1, 1)[:M].contiguous()
    a = A.mx_quantize(X, bits=bits)
    b = A.mx_quantize(X[:64].contiguous(), bits=bits)
    c, d = a.codes.view(torch.uint8), b.codes.view(torch.uint8)
    n = M // 64
    assert torch.equal(c[:64 * n].view(n, 64, -1), d.expand(n, -1, -1)) and torch.equal(c[64 * n:], d[:M - 64 * n])
    c, d = a.scales.view(torch.uint8), b.scales.view(torch.uint8)
    assert torch.equal(c[:64 * n].view(n, 64, -1), d.expand(n, -1, -1)) and torch.equal(c[64 * n:], d[:M - 64 * n])


def test_pack_past_32_bits():
    """Weights of more than 16 GiB, whose codes take more than 4: the last columns pack and unpack as alone."""
    K, N, n = 16384, 64 * 8320 - 7, 64 * 9 - 7
    W = torch.zeros((K, N), dtype=torch.bfloat16, device=DEV)
    assert K * N > 2 ** 33
    tail = torch.randn((K, n), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).bfloat16()
    W[:, -n:] = tail
    q, t = A.mx_pack(W), A.mx_pack(tail)
    del W
    assert torch.equal(q.codes[-9:], t.codes) and torch.equal(q.scales[-9:].view(torch.uint8), t.scales.view(torch.uint8))
    assert t.codes.any() and not q.codes[:-9].any()
    back = A.mx_unpack(q)
    assert torch.equal(back[:, -n:], A.mx_unpack(t)) and not back[:, :-n].any()
