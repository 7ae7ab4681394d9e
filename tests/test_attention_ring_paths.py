"""The plan of the attention for the cases of its tiles' race test, on the host: every tile kernel, with four stages or more."""
import subprocess

from tests.attention_ring_paths import CASES
from tests.test_attention_plan_paths import PATHS, plan  # noqa: F401  (the fixture that builds the printer)


def test_every_tile_kernel_has_four_stages(plan):  # noqa: F811
    text = "".join("%d %d %d %d %d %d\n" % (B, n, -(-L // T) * T, Hq, Hk, D) for B, n, L, Hq, Hk, D, T in CASES)
    out = subprocess.run([plan], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split("\n")
    got = set()
    for (B, n, L, Hq, Hk, D, T), line in zip(CASES, out):
        rows, split, _, _ = map(int, line.split())
        stages = -(-L // (rows // 2))                    # 64 tokens with 128 rows, 128 with 256
        assert stages // split >= 4, (L, rows, split)
        got.add((rows, D, split > 1))
    assert got == {p for p in PATHS if p[0] > 16}
