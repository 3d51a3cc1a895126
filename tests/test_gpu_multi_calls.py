"""Calls for several new tokens that the documentation allows and that are easy
to get wrong."""
import pytest
import torch

import query_aware_sparse_tb_b200 as tb
from test_gpu_multi import i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("row", [771, 773, 1 << 33])
def test_one_token_cut_from_a_buffer_of_any_row_length(row):
    """The stride of a dimension of size 1 says nothing about memory."""
    d, hq, hkv = 64, 8, 2
    width = (hq + 2 * hkv) * d
    flat = torch.randn(width, device=DEV).to(torch.bfloat16)
    qkv = torch.as_strided(flat, (1, width), (row, 1))
    K = torch.zeros(1, hkv, 4, d, dtype=torch.bfloat16, device=DEV)
    V, Q = torch.zeros_like(K), torch.zeros(1, hq, d, dtype=torch.bfloat16, device=DEV)
    ws = tb.workspace(256)
    tb.norm_rope_append(tb.dims(1, hq, hkv, d, 16, 4), qkv, i32([0, 1]), i32([3]), None, None, None, 0.0, None, False,
                        Q, K, V, ws)
    assert tb.workspace_check(ws) == 0
    x = flat.view(hq + 2 * hkv, d)
    assert torch.equal(Q[0], x[:hq]) and torch.equal(K[0, :, 2], x[hq:hq + hkv]) and torch.equal(V[0, :, 2], x[hq + hkv:])
