"""Pins of the MX oracle: the formats' values, rounding at ties, scale bytes, layouts, by hand."""
import numpy as np
import torch

from oracle import mx_oracle as M


def test_element_values():
    t = M.MAGNITUDES[8]
    assert t[0] == 0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[56] == 1.0 and t[126] == 448.0
    assert np.all(np.diff(t) > 0) and len(t) == 127
    ref = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref, t)


def test_rounding_to_nearest_even_and_saturation():
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0, -0.25, -0.0, 0.2501, -100.0])
    assert M.round_codes(v, 4).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 8, 8, 1, 15]
    v = np.array([1.0, 1.0625, 1.1875, 17.0, 19.0, 448.0, 500.0, 2.0 ** -10, 3 * 2.0 ** -10])
    assert M.code_values(M.round_codes(v, 8), 8).tolist() == [1.0, 1.0, 1.25, 16.0, 20.0, 448.0, 448.0, 0.0, 2.0 ** -8]
    x = np.random.default_rng(0).standard_normal(4096) * 100
    ref = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn)
    # torch rounds the float32 of x; these draws are not next to a border
    assert np.array_equal(M.code_values(M.round_codes(x, 8), 8), ref.double().numpy())


def test_scale_bytes():
    p = np.zeros((1, 32))
    assert M.quantize(p, 4)[1][0, 0] == 0
    for top, bits, E in ((6.0, 4, 127), (7.99, 4, 127), (8.0, 4, 128), (3.99, 4, 126), (448.0, 8, 127),
                         (256.0, 8, 127), (255.9, 8, 126), (2.0 ** -130, 4, 0), (2.0 ** -126, 8, 0),
                         (2.0 ** -118, 8, 1), (2.0 ** 127, 4, 252), (2.0 ** 127, 8, 246)):
        p[0, 5] = top
        assert M.quantize(p, bits)[1][0, 0] == E, (top, bits)
    for bad in (np.inf, -np.inf, np.nan):
        p[0, 5] = bad
        c, E = M.quantize(p, 8)
        assert E[0, 0] == 255 and not c.any() and np.isnan(M.values(c, E, 8)).all()


def test_weight_layout_positions():
    assert [M.scale_position(c) for c in (0, 1, 16, 17, 63)] == [0, 4, 1, 5, 63]
    rng = np.random.default_rng(1)
    K, N = 96, 70
    c, E = rng.integers(0, 16, (K, N)).astype(np.uint8), rng.integers(100, 150, (K // 32, N)).astype(np.uint8)
    codes, scales = M.weights_layout(c, E)
    assert codes.shape == (2, 4, 64, 16) and scales.shape == (2, 4, 64)
    assert codes[1, 2, 5, 3] == c[64 + 6, 69] | (c[64 + 7, 69] << 4)
    assert not codes[:, 3].any() and not scales[:, 3].any() and not codes[1, :, 6:].any()
    assert np.array_equal(M.weights_values(codes, scales, K, N), M.values(c.T.copy(), E.T.copy(), 4).T)
