"""The attention's tiles on the LDS-poison debug build (child process of tests/test_gpu_attention_ring_poison.py; AWQ_LIBRARY names
the library): a stage of K and V holds NaN between its last reader and its next writer, so that a read that a missing wait or
barrier lets run early shows.  Prints one line per case; exits non-zero on the first failure."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from tests.attention_ring_paths import CASES  # noqa: E402
from tests.fp8_util import Batch, attend, check_attention, dev  # noqa: E402

for B, n, L, Hq, Hk, D, T in CASES:
    for causal in (True, False):
        print(f"[poison] {B} {n} {L} {Hq} {Hk} {D} {T} {causal}", flush=True)
        batch = Batch([(L - 30 * b, n - 5 * b) for b in range(B)], Hq, Hk, D, T, L)
        if not causal:
            batch.table[0, 3] = -1                       # a hole in the second stage or the first
        batch.upload()
        q = dev(batch.queries())
        check_attention(batch, q, attend(batch, q, causal), causal, label=(B, n, L, Hq, Hk, D, T, causal))
print("[poison] all cases ok", flush=True)
