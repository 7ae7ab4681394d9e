"""The plan of the attention for the calls of tests/attention_kernels.py, on the host."""
import itertools
import subprocess

from tests.attention_kernels import HEADS, MOST_SEQUENCES, WIDE
from tests.test_attention_plan_paths import plan  # noqa: F401  (the fixture that builds the printer)


def test_the_calls_take_the_kernels_that_they_name(plan):  # noqa: F811
    cases = [(n, *WIDE[rows], *heads, D, rows) for n, rows, heads, D in
             itertools.product(range(1, MOST_SEQUENCES + 1), WIDE, HEADS, (64, 128))]
    cases += [(n, 1, tokens, *heads, D, 16) for n, tokens, heads, D in
              itertools.product(range(1, MOST_SEQUENCES + 1), (16, 512, 4096), HEADS, (64, 128))]
    text = "".join("%d %d %d %d %d %d\n" % c[:6] for c in cases)
    out = subprocess.run([plan], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split("\n")
    assert [int(line.split()[0]) for line in out if line] == [c[6] for c in cases]
