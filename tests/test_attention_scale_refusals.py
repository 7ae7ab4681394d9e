"""Scales that the attention refuses, on the host: what the kernels would use, scale * log2 e, has to be finite."""
import ctypes

import pytest

from weight_only_int4_act_amd import awq as A


@pytest.mark.parametrize("scale,refused", [(3.4e38, True), (-3.4e38, True), (2.4e38, True), (1e39, True), (2.3e38, False)])
def test_scale(scale, refused):
    """Every call is rejected before anything is enqueued: the workspace, which is looked at behind the scale, is missing."""
    far = [ctypes.c_void_p(0x100000000 * (i + 1)) for i in range(8)]
    q, cu, length, table, k, v, e, out = far
    got = A.library().awq_attention(q, 5, 8, 2, 64, cu, length, table, 2, 4, 3, k, v, e, 9, 16, ctypes.c_float(scale), 1, out,
                                    None, 0, None)
    assert A.awq_attention_workspace_size(5, 2, 3, 8, 2, 64) > 0
    assert got == (A.AWQ_ERR_INVALID_ARG if refused else A.AWQ_ERR_WORKSPACE)
