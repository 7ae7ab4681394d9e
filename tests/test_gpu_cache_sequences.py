"""Sequences whose counts of rows decrease or leave the rows, on the GPU, for the append (q and the cache) and for the attention,
with norms, a rotation and a cache of its own for each: every row that one sequence has, every token stored and every row
that none has, as each sequence gives them by itself."""
import numpy as np
import pytest
import torch

from tests.fp8_util import A, DEV, Batch, attend, dev
from tests.test_gpu_append import EPS, inputs

pytestmark = pytest.mark.gpu


def batch(cu, lengths, Hq, Hk, D, T, seed, rows):
    B = Batch([(L, 1) for L in lengths], Hq, Hk, D, T, seed)
    B.cu, B.M = np.asarray(cu, np.int32), rows
    B.max_q = rows
    B.upload()
    return B


def step(B, x, cu, b=None):
    """q and the attention, causal and not, of all sequences or of sequence b alone, over B's cache."""
    d = dict(B.d, cu=torch.tensor(cu, dtype=torch.int32, device=DEV))
    if b is not None:
        d.update(length=d["length"][b:b + 1].clone(), table=d["table"][b:b + 1].contiguous())
    q = torch.full((B.M, B.Hq, B.D), 7.0, dtype=torch.bfloat16, device=DEV)
    A.awq_qkv_append(dev(x["qkv"]), dev(x["qw"]), dev(x["kw"]), EPS, torch.from_numpy(x["rope"]).to(DEV), False, d["cu"],
                     d["length"], d["table"], B.max_q, q, d["k"], d["v"], d["E"])
    outs = []
    for causal in (True, False):
        out = torch.full_like(q, 7.0)
        n = d["length"].shape[0]
        ws = A.workspace(A.awq_attention_workspace_size(B.M, n, B.max_q, B.Hq, B.Hk, B.D), DEV)
        A.awq_attention(q, d["cu"], d["length"], d["table"], B.max_q, d["k"], d["v"], d["E"], B.D ** -0.5, causal, out, ws)
        outs.append(out)
    return q, *outs


CASES = [
    # a count below the one before; one that rises but stays below; one below the first; bounds outside the rows
    ([0, 9, 4, 20], [40, 30, 50]), ([0, 10, 3, 6, 25], [33, 20, 40, 60]), ([5, 3, 12, 2, 30], [20, 50, 20, 70]),
    ([-4, 50, 30, 1000], [60, 10, 90]),
]


@pytest.mark.parametrize("cu,lengths", CASES)
@pytest.mark.parametrize("Hq,Hk,D,T", [(2, 2, 64, 16), (8, 1, 128, 64), (32, 2, 64, 128)])
def test_counts_that_decrease(cu, lengths, Hq, Hk, D, T):
    rows = 70
    B = batch(cu, lengths, Hq, Hk, D, T, 1, rows)
    x = inputs(B, D, True, P=max(lengths))
    got, cache = step(B, x, cu), B.download()
    owners = np.zeros(rows, int)
    want = [np.zeros((rows, Hq, D)) for _ in got]
    B.upload()
    for b in range(len(lengths)):
        r = slice(min(max(cu[b], 0), rows), min(max(cu[b + 1], 0), rows))
        owners[r] += 1
        for w, t in zip(want, step(B, x, [cu[b], cu[b + 1]], b)):
            w[r] = t.float().cpu().numpy()[r]
    for a, b in zip(cache, B.download()):
        assert np.array_equal(a, b)
    # rounding of p and the order of sums may differ with the number of sequences, which choose the kernel: two halves of
    # a step of bf16, 2^-7 of the result, and p's rounding on both sides, 2^-7 of the largest |v| (448 2^(120 - 127) = 3.5, and
    # normal numbers below 5), with as much as is left to 7 for the float32 sums
    for name, t, w in zip(("q", "causal", "not causal"), got, want):
        t = t.float().cpu().numpy()
        near = np.abs(t - w) <= (0 if name == "q" else 2.0 ** -7 * (np.abs(w) + 7))
        assert near[owners == 1].all(), (name, np.argwhere(~near)[:4])
        assert (t[owners == 0] == 7).all(), name


def test_a_decrease_leaves_a_sequence_without_rows():
    """And the one behind it, which begins where rows are free, with its own."""
    B = Batch([(40, 12), (33, 0), (50, 8)], 4, 2, 64, 16, 3)
    B.upload()
    clean = attend(B, q := dev(B.queries()))
    B.d["cu"] = torch.tensor([12, 0, 0, 8], dtype=torch.int32, device=DEV)    # none, none, rows 0 .. 7
    out = attend(B, q)
    B.d["cu"] = torch.tensor([0, 0, 0, 8], dtype=torch.int32, device=DEV)
    assert torch.equal(out, attend(B, q)) and (out[8:] == 7).all() and not torch.equal(out, clean)
