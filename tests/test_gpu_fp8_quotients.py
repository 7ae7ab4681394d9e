"""Elements of the 8-bit groups of 128 on the GPU, code for code: the float32 quotient p / s rounded to e4m3, for numbers of
every mantissa under scales of every mantissa that bf16 has, where many quotients lie on or next to a border of two codes."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.fp8_util import A, bf16, dev, f32, u8

pytestmark = pytest.mark.gpu
EXPONENTS = [-125, -110, -104, -103, -48, -33, -32, -31, -30, -1, 0, 60, 127]   # of a group's largest number


def groups(e: int) -> np.ndarray:
    """[R, 128] bf16 numbers: the first of a row its largest, of every mantissa at 2^e; the others of every mantissa and sign
    down to 2^-21 of it, where elements end."""
    m = 1 + np.arange(128) / 128
    down = np.arange(22)
    p = np.broadcast_to((m[None, :] * 2.0 ** -down[:, None]).reshape(1, -1), (128, 22 * 128)) * 2.0 ** e
    top = m[:, None] * 2.0 ** e
    p = np.where(p > top, top, p) * np.where(np.arange(p.shape[1]) % 3 == 1, -1, 1)
    p = np.concatenate((p, np.zeros((128, 127 - p.shape[1] % 127)), -np.zeros((128, 127))), 1).reshape(-1, 127)
    return f32(bf16(np.concatenate((np.repeat(top, p.shape[0] // 128, 0), p), 1))).astype(np.float64)


def elements(p: np.ndarray, s: np.ndarray) -> np.ndarray:
    """Both have at most 24 significant bits, so the float64 quotient (53 >= 2 * 24 + 2) rounds to the same float32 as the
    exact one."""
    return O.codes_of((p / s.astype(np.float64)[:, None]).astype(np.float32).astype(np.float64))


def check(codes, scales, p, label):
    s = O.scale_of(np.abs(p).max(1))
    assert np.array_equal(scales, s), label
    want = elements(p, s)
    bad = codes != want
    assert not bad.any(), (label, int(bad.sum()), bad.size, p[bad][:4], codes[bad][:4], want[bad][:4])


def test_the_cases_hold_what_they_are_for():
    """Products with the rounded reciprocal give other codes here."""
    p = groups(0)
    s = O.scale_of(np.abs(p).max(1))
    r = (np.float32(1) / s)[:, None]
    other = O.codes_of((p.astype(np.float32) * r).astype(np.float64))
    assert (other != elements(p, s)).sum() > 100


@pytest.mark.parametrize("e", EXPONENTS)
def test_quantize(e):
    p = groups(e)
    a = A.fp8_quantize(dev(bf16(p)))
    torch.cuda.synchronize()
    check(u8(a.codes), a.scales.cpu().numpy()[:, 0], p, e)


@pytest.mark.parametrize("e", EXPONENTS)
def test_pack(e):
    """A row's numbers as one column of a group of weights whose other columns hold nothing larger."""
    p = groups(e)[::37]
    R = p.shape[0]
    W = np.zeros((128, 128 * R))
    W[:, 128 * np.arange(R) + np.arange(R) % 128] = p.T
    q = A.fp8_pack(dev(bf16(W)))
    torch.cuda.synchronize()
    got = O.weights_codes(u8(q.codes), 128, 128 * R)[:, 128 * np.arange(R) + np.arange(R) % 128]
    check(got.T, q.scales.cpu().numpy()[:, 0], p, e)
