"""max_q outside 32 bits, on the host: the foreign calls would take its low 32 bits, leave rows out and size the workspace for
those."""
import pytest
import torch

from weight_only_int4_act_amd import awq as A


@pytest.mark.parametrize("max_q", [-(1 << 32) + 5, -(1 << 31) - 1, 1 << 31, (1 << 32) + 5, (1 << 64) + 1])
def test_refused(max_q):
    bf, i32 = torch.bfloat16, torch.int32
    k, v, e = (torch.zeros(5, 2, *s, dtype=torch.uint8) for s in ((16, 64), (1, 64, 16), (2,)))
    q, qkv = torch.zeros(4, 4, 64, dtype=bf), torch.zeros(4, 8 * 64, dtype=bf)
    seqs = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=i32), max_q
    with pytest.raises(ValueError, match="max_q"):
        A.awq_qkv_append(qkv, None, None, 1e-5, None, False, *seqs, q, k, v, e)
    with pytest.raises(ValueError, match="max_q"):
        A.awq_attention(q, *seqs, k, v, e, 0.1, True, q.clone(), None)
    assert A.awq_attention_workspace_size(4, 2, max_q, 4, 2, 64) == 0


@pytest.mark.parametrize("at", range(1, 6))
def test_sizes_past_32_bits_have_no_workspace(at):
    ok = [4, 2, 3, 4, 2, 64]
    assert A.awq_attention_workspace_size(*ok) > 0
    for off in (1 << 32, -(1 << 32)):
        assert A.awq_attention_workspace_size(*(v + off if i == at else v for i, v in enumerate(ok))) == 0
