"""Calls for several new tokens that the documentation allows and that are easy
to get wrong."""
import pytest
import torch

import query_aware_sparse_tb_b200 as tb
import test_gpu_multi as multi
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


# ------------------------------------------------------------------ acceptance

def accept_case(lens_of, n, T, path, caches_of, cap=64, hkv=2, d=64, layers=3):
    kv = torch.randn(layers, 2, len(n), hkv, cap, d, device=DEV).to(torch.bfloat16)
    caches = torch.tensor(caches_of([[kv[l, i].data_ptr() for i in range(2)] for l in range(layers)]), dtype=torch.int64,
                          device=DEV)
    before, new_len, ws = kv.clone(), torch.full((len(n),), -7, dtype=torch.int32, device=DEV), tb.workspace(256)
    tb.tree_accept(tb.dims(len(n), 4 * hkv, hkv, d, 16, cap), caches.numel() // 2, caches, i32(multi.starts(n)), i32(T),
                   i32(path), i32(lens_of), new_len, ws)
    want = before.clone()
    for b, k in enumerate(lens_of):
        base = T[b] - n[b]
        if k:
            want[:, :, b, :, base:base + k] = before[:, :, b, :, [base + j for j in path[b][:k]]]
    return kv, want, new_len.tolist(), tb.workspace_check(ws)


def test_accept_does_not_look_at_idle_sequences():
    """A sequence without drafted tokens is not looked at, whatever its length
    says; its length comes back as it is."""
    n, T = [4, 0, 0, 0, 3], [20, -1, 0, 1 << 30, 9]
    kv, want, new_len, flags = accept_case([2, 0, 0, 0, 1], n, T, [[1, 3], [0, 0], [5, 5], [0, 0], [2, 0]],
                                           lambda a: [x for pair in a for x in pair])
    assert flags == 0 and new_len == [18, -1, 0, 1 << 30, 7]
    assert torch.equal(kv, want)


@pytest.mark.parametrize("caches_of", [
    lambda a: [x for pair in a for x in pair] + a[1],                 # a layer that reads another's cache
    lambda a: [a[0][0], a[0][0], a[0][1], a[0][1]] + a[1] + a[2],     # K and V one array
    lambda a: (a[0] + a[1] + a[2]) * 40,                              # many times
])
def test_accept_moves_a_cache_that_is_listed_twice_once(caches_of):
    n, T = [26, 40], [50, 64]
    path = [list(range(1, 26, 2)) + [0] * 8, list(range(19, 40))]
    for _ in range(5):
        kv, want, new_len, flags = accept_case([13, 21], n, T, path, caches_of)
        assert flags == 0 and new_len == [37, 45]
        assert torch.equal(kv, want)
