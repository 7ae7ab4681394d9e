"""Every kernel of the attention over the cache on the GPU against float64: the cases of tests/attention_paths.py, causal and
not."""
import pytest

from tests.attention_paths import CASES
from tests.fp8_util import Batch, attend, check_attention, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", CASES)
def test_every_kernel(case):
    B, n, L, Hq, Hk, D, T = case
    # the first sequence has L tokens and n new ones, the others fewer
    lengths = [(max(L - 37 * b, 1), max(min(n - 5 * b, L - 37 * b), 1)) for b in range(B)]
    batch = Batch(lengths, Hq, Hk, D, T, L)
    batch.upload()
    q = dev(batch.queries())
    for causal in (True, False):
        check_attention(batch, q, attend(batch, q, causal), causal, label=(case, causal))
