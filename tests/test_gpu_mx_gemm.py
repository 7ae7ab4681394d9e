"""The MX product on the GPU against float64 products of the values its operands stand for, within the
bound that float32 accumulation and one bf16 rounding leave."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as O
from tests.mx_util import A, DEV, check_product, product, random_acts, random_weights

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32, 8), (1, 128, 64), (1, 8192, 1024), (2, 96, 72), (3, 160, 200), (7, 4096, 520), (13, 2080, 136),
          (16, 512, 4096), (17, 1024, 64), (31, 352, 328), (33, 512, 512), (64, 224, 1032), (65, 1152, 256),
          (127, 128, 136), (129, 1056, 264), (200, 608, 520), (256, 512, 512), (257, 2048, 776), (300, 4096, 1024),
          (513, 96, 264), (1030, 736, 1288)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(M, K, N, bits):
    xc, xs, x = random_acts(M, K, bits, M + K + N)
    wc, wsc, w = random_weights(K, N, M + K + N + 1)
    check_product(product(xc, xs, wc, wsc, M, K, N), x, w, bits, (M, K, N, bits))


# 128- and 256-row tiles, with and without a split of K, scales that start on a 4-byte boundary (K a multiple
# of 128) and that do not, an odd number of 128-channel chunks, ragged rows and columns
LARGE = [(2459, 224, 1568), (2390, 640, 1560), (1800, 608, 4432), (1576, 384, 6776), (340, 4960, 5560),
         (388, 5760, 4976), (1659, 7648, 2440), (2345, 8576, 1552), (111, 4288, 16), (84, 4352, 16), (27, 6656, 8),
         (1576, 736, 6776), (1576, 1024, 6776), (1576, 1152, 6776), (1576, 1280, 6776)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", LARGE)
def test_product_in_large_tiles(M, K, N, bits):
    xc, xs, x = random_acts(M, K, bits, M + K + N)
    wc, wsc, w = random_weights(K, N, M + K + N + 1)
    check_product(product(xc, xs, wc, wsc, M, K, N), x, w, bits, (M, K, N, bits))


# K cut into slices, up to sixteen, in the register kernel and in tiles of 64, 128 and 256 rows; slices of four
# chunks and more, of which the last has one to four; and 128-row tiles of four and twelve chunks
SPLIT = [(5, 25056, 72), (20, 24000, 8), (40, 11008, 8), (60, 6848, 8), (70, 11008, 264), (70, 11040, 264),
         (150, 6176, 8), (2000, 16416, 520), (2000, 16512, 520), (2000, 17888, 2056), (2000, 17920, 2056),
         (2390, 512, 1560), (2390, 1504, 1560)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", SPLIT)
def test_product_in_slices(M, K, N, bits):
    xc, xs, x = random_acts(M, K, bits, M + K + N)
    wc, wsc, w = random_weights(K, N, M + K + N + 1)
    check_product(product(xc, xs, wc, wsc, M, K, N), x, w, bits, (M, K, N, bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("M,K,N", [(5, 256, 64), (70, 512, 128), (1600, 384, 6776)])
def test_scales_at_any_address(M, K, N, bits, offset):
    """Scales of the activations that start 1 to 3 bytes past a 4-byte boundary: the same bits."""
    xc, xs, _ = random_acts(M, K, bits, 1)
    wc, wsc, _ = random_weights(K, N, 2)
    room = torch.full((xs.numel() + 8,), 0xFF, dtype=torch.uint8, device=DEV)
    moved = room[offset:offset + xs.numel()].view(M, -1)
    moved.copy_(xs)
    a, b = product(xc, xs, wc, wsc, M, K, N), product(xc, moved, wc, wsc, M, K, N)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 512), (5, 1024, 192), (40, 1120, 256), (300, 512, 520), (600, 1024, 776), (1800, 512, 4440), (2390, 160, 1560)])
def test_integers_are_exact(M, K, N, bits):
    """Elements that are small integers under scales of 1: every partial sum is a float32 integer, so the
    product is the bf16 rounding of the exact one, whatever the order of its sums."""
    rng = np.random.default_rng(M)
    x, w = rng.integers(-3, 4, (M, K)).astype(np.float64), rng.integers(-3, 4, (K, N)).astype(np.float64)
    E = np.full((M, K // 32), 127, np.uint8)
    c = O.round_codes(x, bits)
    t = torch.from_numpy(c if bits == 8 else O.pair(c))
    xc = (t.view(torch.float8_e4m3fn) if bits == 8 else t).to(DEV)
    wc, wsc = (torch.from_numpy(a).to(DEV) for a in O.weights_layout(O.round_codes(w, 4), np.full((K // 32, N), 127, np.uint8)))
    Y = product(xc, torch.from_numpy(E).to(DEV), wc, wsc, M, K, N)
    assert torch.equal(Y.cpu(), torch.from_numpy((x @ w).astype(np.float32)).to(torch.bfloat16))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", [(1, 256, 128), (6, 1024, 72), (100, 384, 264), (400, 512, 520), (1800, 544, 4432), (2390, 160, 1560)])
def test_one_element_at_a_time(M, K, N, bits):
    """Each row of x has one nonzero element, with its block's own scale: row m of Y is one row of W times a
    power of two, exactly.  A block or a scale taken from another place shows."""
    rng = np.random.default_rng(K)
    k = rng.integers(0, K, M)
    c = np.zeros((M, K), np.uint8)
    c[np.arange(M), k] = O.round_codes(np.ones(M), bits)
    E = rng.integers(120, 134, (M, K // 32)).astype(np.uint8)
    t = torch.from_numpy(c if bits == 8 else O.pair(c))
    xc = (t.view(torch.float8_e4m3fn) if bits == 8 else t).to(DEV)
    wc, wsc, w = random_weights(K, N, K)
    Y = product(xc, torch.from_numpy(E).to(DEV), wc, wsc, M, K, N)
    ref = w[k] * 2.0 ** (E[np.arange(M), k // 32] - 127.0)[:, None]
    assert torch.equal(Y.cpu().float(), torch.from_numpy(ref.astype(np.float32)))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", [(1, 1024, 128), (20, 256, 64), (300, 640, 264), (1800, 608, 4432), (2390, 160, 1560)])
def test_nan_blocks_and_extreme_scales(M, K, N, bits):
    xc, xs, _ = random_acts(M, K, bits, 1)
    wc, wsc, _ = random_weights(K, N, 2)
    E = xs.cpu().numpy().copy()
    F = wsc.cpu().numpy().copy()
    if M > 2:
        E[1, 0], E[2, -1] = 0, 0                 # the smallest scale
        E[M // 2, K // 64] = 255                 # a row of NaN
    F[0, 1, O.scale_position(5)] = 255           # a column of NaN
    F[0, 0, O.scale_position(9)] = 0
    F[0, 2, O.scale_position(9)] = 200
    c = xc.view(torch.uint8).cpu().numpy()
    x = O.values(c if bits == 8 else O.unpair(c), E, bits)
    w = O.weights_values(wc.cpu().numpy(), F, K, N)
    Y = product(xc, torch.from_numpy(E).to(DEV), wc, torch.from_numpy(F).to(DEV), M, K, N)
    check_product(Y, x, w, bits, (M, K, N, bits))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,K,N", [(1, 1024, 136), (9, 96, 72), (70, 128, 200), (300, 512, 264), (130, 96, 72), (1800, 608, 4432), (2459, 160, 1568)])
def test_nothing_else_is_written_or_read(M, K, N, bits):
    """Y lies between guard rows; the activations are followed by NaN codes and NaN scales, which no row
    may see (K = 96 ends inside a 128-channel chunk)."""
    xc, xs, x = random_acts(M, K, bits, 4)
    wc, wsc, w = random_weights(K, N, 5)
    nb = xc.view(torch.uint8).numel()
    big = torch.full((nb + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    big[:nb] = xc.view(torch.uint8).reshape(-1)
    bs = torch.full((xs.numel() + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    bs[:xs.numel()] = xs.reshape(-1)
    xc = big[:nb].view(M, -1)
    xc = xc.view(torch.float8_e4m3fn) if bits == 8 else xc
    Yg = torch.full((M * N + 2048,), 3.0, dtype=torch.bfloat16, device=DEV)
    Y = Yg[1024:1024 + M * N].view(M, N)
    ws = A.workspace(A.awq_mx_gemm_workspace_size(M, K, N, bits), DEV)
    A.awq_mx_gemm(xc, bs[:xs.numel()].view(M, -1), wc, wsc, Y, ws)
    torch.cuda.synchronize()
    assert (Yg[:1024] == 3).all() and (Yg[1024 + M * N:] == 3).all()
    check_product(Y, x, w, bits, (M, K, N, bits))


@pytest.mark.parametrize("bits", [8, 4])
def test_repeated_calls_agree_on_one_workspace(bits):
    """One workspace for every shape in turn, three rounds: equal bits each time, counters left at zero."""
    shapes = [(1, 8192, 1024), (13, 4096, 520), (64, 2048, 256), (300, 1024, 776), (1, 1024, 64), (129, 4096, 264),
              (340, 4960, 5560), (30, 2240, 8), (1800, 608, 4432)]
    ops = [(random_acts(M, K, bits, i)[:2], random_weights(K, N, i)[:2]) for i, (M, K, N) in enumerate(shapes)]
    ws = A.workspace(max(A.awq_mx_gemm_workspace_size(*s, bits) for s in shapes), DEV)
    first = None
    for _ in range(3):
        ys = [product(*a, *b, *s, ws=ws) for s, (a, b) in zip(shapes, ops)]
        assert not ws[:65536].any()
        if first is None:
            first = ys
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(first, ys))


def test_rows_do_not_depend_on_their_neighbours():
    """A row's result is the same bits alone in a batch of the same plan, wherever it stands."""
    M, K, N = 300, 1024, 264
    for bits in (8, 4):
        xc, xs, _ = random_acts(M, K, bits, 1)
        wc, wsc, _ = random_weights(K, N, 2)
        Y = product(xc, xs, wc, wsc, M, K, N)
        p = torch.randperm(M, generator=torch.Generator().manual_seed(0)).to(DEV)
        xp = xc.view(torch.uint8)[p].contiguous()
        Z = product(xp.view(xc.dtype), xs[p].contiguous(), wc, wsc, M, K, N)
        assert torch.equal(Y[p].view(torch.int16), Z.view(torch.int16))


def small_integers(M, K, bits, seed):
    """Activations -2 .. 2 under scales of 1 (every sum of up to 2^19 products with e2m1 elements is exact)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randint(-2, 3, (M, K), device=DEV, generator=g, dtype=torch.int8)
    E = torch.full((M, K // 32), 127, dtype=torch.uint8, device=DEV)
    if bits == 8:
        return v.to(torch.float8_e4m3fn), E
    c = torch.where(v < 0, 8, 0).to(torch.uint8) | (v.abs().to(torch.uint8) << 1)     # 1 -> 2, 2 -> 4
    return c[:, ::2] | (c[:, 1::2] << 4), E


def test_weights_past_32_bits():
    """Codes of more than 4 GiB: the last columns of a product equal those of their tiles alone."""
    K, N = 16384, 64 * 8320
    g = torch.Generator(device=DEV).manual_seed(1)
    wc = torch.zeros((N // 64, K // 32, 64, 16), dtype=torch.uint8, device=DEV)
    assert wc.numel() > 2 ** 32
    wc[-9:] = torch.randint(0, 256, wc[-9:].shape, dtype=torch.uint8, device=DEV, generator=g)
    ws = torch.full((N // 64, K // 32, 64), 127, dtype=torch.uint8, device=DEV)
    for M, bits in ((1, 8), (70, 4), (300, 8)):
        xc, xs = small_integers(M, K, bits, M)
        Y = product(xc, xs, wc, ws, M, K, N)
        Z = product(xc, xs, wc[-9:].contiguous(), ws[-9:].contiguous(), M, K, 576)
        assert torch.equal(Y[:, -576:], Z) and Z.any() and not Y[:, :-576].any()


@pytest.mark.parametrize("bits", [8, 4])
def test_rows_past_32_bits(bits):
    """Activations, and then a result, of more than 4 GiB: the last rows equal those of a product of their own."""
    wc, ws, _ = random_weights(16384, 8, 3)
    ws.fill_(127)
    M = 2 ** 32 * 8 // bits // 16384 + 70
    xc, xs = small_integers(64, 16384, bits, 4)
    big = torch.zeros((M, xc.shape[1]), dtype=torch.uint8, device=DEV)
    big[-64:] = xc.view(torch.uint8)
    E = torch.full((M, 512), 127, dtype=torch.uint8, device=DEV)
    Y = product(big.view(xc.dtype), E, wc, ws, M, 16384, 8)
    assert torch.equal(Y[-64:], product(xc, xs, wc, ws, 64, 16384, 8)) and not Y[:-64].any() and Y[-64:].any()
    del big, E
    M, N = 4099, 64 * 8320
    wc = torch.randint(0, 256, (N // 64, 4, 64, 16), dtype=torch.uint8, device=DEV,
                       generator=torch.Generator(device=DEV).manual_seed(5))
    wc[:, 3:] = 0                                # past K
    ws = torch.full((N // 64, 4, 64), 127, dtype=torch.uint8, device=DEV)
    ws[:, 3:] = 0
    xc, xs = small_integers(M, 96, bits, 6)
    Y = product(xc, xs, wc, ws, M, 96, N)
    assert Y.numel() * 2 > 2 ** 32
    assert torch.equal(Y[-64:], product(xc[-64:].contiguous(), xs[-64:].contiguous(), wc, ws, 64, 96, N)) and Y[-64:].any()
