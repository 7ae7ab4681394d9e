"""Products and norms of the microscaled operators on the LDS-poison debug build (child process of
tests/test_gpu_mx_lds_poison.py; AWQ_LIBRARY names the library): every pipelined LDS buffer holds NaN
codes or scales of about 2^120 between its last reader and its next writer, so that a read that a
missing wait or barrier lets run early shows.  Prints one line per case; exits non-zero on the first
failure."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402

from oracle import mx_oracle as O  # noqa: E402
from tests.mx_util import A, bf16, check_product, check_quantized, dev, f32, product, random_acts, random_weights, rows  # noqa: E402

for bits in (8, 4):
    for M, K, N in ((1, 4096, 256), (13, 2080, 136), (30, 2240, 8), (48, 1024, 264), (64, 224, 1032), (130, 1056, 264),
                    (300, 4096, 1024), (2390, 640, 1560), (1800, 608, 4432), (1576, 1152, 6776), (340, 4960, 5560), (70, 4640, 264),
                    (2390, 1504, 1560)):
        print(f"[poison] product {M} {K} {N} {bits}", flush=True)
        xc, xs, x = random_acts(M, K, bits, M)
        wc, wsc, w = random_weights(K, N, N)
        check_product(product(xc, xs, wc, wsc, M, K, N), x, w, bits, (M, K, N, bits))
    for M, K in ((1, 8192), (700, 2048), (3, 40032)):
        print(f"[poison] norm {M} {K} {bits}", flush=True)
        X, w = rows(M, K, 1), bf16(np.linspace(0.5, 1.5, K))
        a, _ = A.rms_norm(dev(X), dev(w), bits=bits)
        y = O.rms_norm(f32(X).astype(np.float64), None, f32(w).astype(np.float64), 1e-5)
        check_quantized(a.codes, a.scales, y, 8 * 2.0 ** -24, (M, K, bits))
print("[poison] all cases ok", flush=True)
