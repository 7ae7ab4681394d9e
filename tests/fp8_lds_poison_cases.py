"""The 8-bit operators on the LDS-poison debug build (child process of tests/test_gpu_fp8_lds_poison.py; AWQ_LIBRARY
names the library): LDS holds NaN before its first writer and, in the product's pipeline, between a place's last reader
and its next writer, so that a read that a missing wait or barrier lets run early shows.  Prints one line per
case; exits non-zero on the first failure."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

from tests import test_gpu_append as P  # noqa: E402
from tests.fp8_paths import CASES  # noqa: E402
from tests.fp8_util import (A, DEV, Batch, attend, bf16, check_attention, check_product, dev, product, random_acts,  # noqa: E402
                            random_weights)

for M, K, N in [*CASES, (1, 4096, 264), (64, 640, 256), (300, 4112, 1032), (2390, 1504, 1560)]:
    print(f"[poison] product {M} {K} {N}", flush=True)
    xc, xs, x = random_acts(M, K, M)
    wc, ws, w = random_weights(K, N, N)
    check_product(product(xc, xs, wc, ws, N), torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV), (M, K, N))
for K, N in ((16, 1), (656, 200), (1024, 333)):
    print(f"[poison] pack {K} {N}", flush=True)
    W = dev(bf16(np.random.default_rng(K).standard_normal((K, N)).astype(np.float32)))
    q = A.fp8_pack(W)
    c = q.codes.double().view(-1, q.codes.shape[1], 4, 2, 4, 16, 16).permute(1, 3, 4, 6, 0, 2, 5)
    w = c.reshape(q.codes.shape[1] * 128, -1)[:K, :N]
    w = w * q.scales.double().t().repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]
    # a code is off by half a step, 2^-4 of the number or 2^-10 of the group's scale, and 2 units in the last place
    bound = W.double().abs() * (2.0 ** -4 + 2.0 ** -21) + 2.0 ** -9 * W.double().abs().max() / 448
    assert ((w - W.double()).abs() <= bound).all(), (K, N)
for D in (64, 128):
    for T in (16, 32, 64, 128):
        for lengths in ([(1, 1), (40, 1), (200, 1), (1031, 1)], [(130, 130), (300, 33), (90, 2)], [(700, 300)]):
            print(f"[poison] cache {lengths} {D} {T}", flush=True)
            B = Batch(lengths, 8, 2, D, T, 1)
            B.upload()
            q = dev(B.queries())
            check_attention(B, q, attend(B, q), label=(lengths, D, T))
            x = P.inputs(B, D, True)
            P.check(B, x, P.append(B, x), label=(lengths, D, T))
print("[poison] all cases ok", flush=True)
