"""Pins of the 8-bit oracle: scales, layouts, scale bytes of the cache, rotation and attention, by hand."""
import numpy as np

from oracle import fp8_oracle as O


def test_scales_of_groups():
    assert O.scale_of(np.array([448.0]))[0] == 1 and O.scale_of(np.array([0.0]))[0] == 2.0 ** -120
    assert np.isnan(O.scale_of(np.array([np.inf]))[0])
    p = np.zeros((2, 130))
    p[0, 5], p[0, 129], p[1, 3] = -7, 3, np.nan
    assert O.group_top(p).tolist() == [[7, 3], [np.inf, 0]]
    W = np.zeros((130, 129))
    W[1, 2], W[129, 128] = -5, 6
    assert O.weight_top(W).tolist() == [[5, 0], [0, 6]]


def test_weights_layout():
    c = np.random.default_rng(0).integers(0, 126, (144, 70)).astype(np.uint8)
    w = O.weights_layout(c)
    assert w.shape == (2, 2, 8, 64, 16) and np.array_equal(O.weights_codes(w, 144, 70), c)
    # channel 64 + 16 + 3 of column 16 * 2 + 5: f = 2, h = 1, g = 1, i = 5, byte 3
    assert w[0, 0, 5, 21, 3] == c[83, 37] and not w[1, :, :, 6:16].any()
    # the checkpoint's codes [N, K] by the permutation that the header names
    z = np.zeros((128, 256), np.uint8)
    z[:70, :144] = c.T
    assert np.array_equal(z.reshape(2, 4, 16, 2, 2, 4, 16).transpose(0, 3, 1, 4, 5, 2, 6).reshape(w.shape), w)


def test_scale_bytes_of_the_cache():
    for top, E in ((0.0, 0), (448.0, 127), (448.1, 128), (449.0, 128), (224.0, 126), (1.75, 119), (1.76, 120),
                   (2.0 ** -130, 0), (3e38, 247), (np.inf, 255), (np.nan, 255)):
        assert O.cache_byte(top) == E, top


def test_v_layout():
    v = np.random.default_rng(1).integers(0, 255, (2, 3, 32, 64)).astype(np.uint8)
    w = O.v_layout(v)
    assert w.shape == (2, 3, 2, 64, 16) and w[1, 2, 1, 7, 5] == v[1, 2, 21, 7] and np.array_equal(O.v_rows(w), v)


def test_rotation_and_attention():
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    turn = np.array([[0.0, 0.0, 1.0, 1.0]])                    # a quarter turn: (a, c) -> (-c, a)
    assert O.rotate(x, turn, 4, False)[0].ravel().tolist() == [-3, -4, 1, 2]
    assert O.rotate(x, turn, 4, True)[0].ravel().tolist() == [-2, 1, -4, 3]
    assert O.rotate(x, np.array([[0.0, 1.0]]), 2, False)[0].ravel().tolist() == [-2, 1, 3, 4]
    k, v = np.zeros((3, 2)), np.array([[1.0, 0], [2, 0], [6, 0]])
    out, size, reach = O.attention(np.ones((2, 2)), k, v, True, 1.0)
    assert out[:, 0].tolist() == [1.5, 3.0] and reach == 0 and np.array_equal(out, size)
    assert O.attention(np.ones((2, 2)), k, v, False, 1.0)[0][:, 0].tolist() == [3.0, 3.0]
    assert O.attention(np.ones((5, 2)), k, v, True, 1.0)[0][:, 0].tolist() == [0, 0, 1, 1.5, 3]
