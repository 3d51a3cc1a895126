"""Refusals of the calls that take several new tokens of a sequence at once,
without a GPU: the C side rejects bad arguments before any CUDA call, the
binding what the C side cannot see."""
import ctypes

import pytest
import torch

from query_aware_sparse_tb_b200 import _lib, build

FAKE = 1 << 20          # 16-byte aligned, never dereferenced: validation fails first
FAR = [FAKE + (i << 36) for i in range(16)]  # far apart: no two arrays overlap


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _d(**kw):
    base = dict(batch=2, n_q_heads=32, n_kv_heads=8, head_dim=128, d_proj=0, ctx_cap=4096)
    base.update(kw)
    return _lib.TbDims(*[base[k] for k in ("batch", "n_q_heads", "n_kv_heads", "head_dim", "d_proj", "ctx_cap")])


BAD_DIMS = [
    (dict(batch=0), "INVALID_ARG"), (dict(ctx_cap=0), "INVALID_ARG"), (dict(n_q_heads=30), "INVALID_ARG"),
    (dict(n_q_heads=24), "UNSUPPORTED"), (dict(n_q_heads=256), "UNSUPPORTED"), (dict(head_dim=96), "UNSUPPORTED"),
    (dict(batch=65536), "UNSUPPORTED"), (dict(ctx_cap=(1 << 22) + 1), "UNSUPPORTED"),
]


def _status(name):
    return getattr(_lib, "TB_ERR_" + name)


def _attn(lib, tree, dims=None, Q=FAR[0], K=FAR[1], V=FAR[2], qb=FAR[3], n=10, mx=5, ctx=FAR[4], mask=FAR[5],
          scale=0.1, out=FAR[6], ws=FAR[7], ws_bytes=1 << 34):
    d = dims or _d()
    if tree:
        return lib.tb_tree_attn(ctypes.byref(d), Q, K, V, qb, n, mx, ctx, mask, scale, out, ws, ws_bytes, None)
    return lib.tb_prompt_attn(ctypes.byref(d), Q, K, V, qb, n, mx, ctx, scale, out, ws, ws_bytes, None)


@pytest.mark.parametrize("tree", [False, True])
def test_attention_refuses(lib, tree):
    for kw, name in BAD_DIMS:
        assert _attn(lib, tree, _d(**kw)) == _status(name), kw
    need = (lib.tb_tree_attn_workspace_bytes if tree else lib.tb_prompt_attn_workspace_bytes)(ctypes.byref(_d()), 10, 5)
    assert need >= 256
    assert _attn(lib, tree, ws_bytes=need - 1) == _lib.TB_ERR_WORKSPACE
    for kw in (dict(Q=0), dict(K=FAKE + 8), dict(V=0), dict(qb=0), dict(qb=FAKE + 2), dict(ctx=0), dict(out=0),
               dict(out=FAKE + 4), dict(ws=0), dict(mx=0), dict(n=-1), dict(scale=0.0), dict(scale=-0.1),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _attn(lib, tree, **kw) == _lib.TB_ERR_INVALID_ARG, kw
    # the result over an input (or a part of one)
    for kw in (dict(out=FAR[0]), dict(out=FAR[1] + 4096), dict(out=FAR[2] - 64)):
        assert _attn(lib, tree, **kw) == _lib.TB_ERR_INVALID_ARG and b"overlaps" in lib.tb_last_error(), kw
    assert _attn(lib, tree, _d(batch=1024, n_kv_heads=8, ctx_cap=1 << 18)) == _lib.TB_ERR_UNSUPPORTED  # 2^31 rows
    if tree:
        assert _attn(lib, tree, mask=0) == _lib.TB_ERR_INVALID_ARG
        assert _attn(lib, tree, mx=1025) == _lib.TB_ERR_UNSUPPORTED
        assert lib.tb_tree_attn_workspace_bytes(ctypes.byref(_d()), 10, 1025) == 0
    # nothing to do is no error, whatever the (empty) arrays' addresses
    assert _attn(lib, tree, n=0, Q=0, out=0) == _lib.TB_OK
    size = lib.tb_tree_attn_workspace_bytes if tree else lib.tb_prompt_attn_workspace_bytes
    assert size(ctypes.byref(_d(head_dim=96)), 10, 5) == 0 and size(ctypes.byref(_d()), -1, 5) == 0


def _rope(lib, dims=None, qkv=FAR[0], stride=48 * 128, qb=FAR[1], n=10, ctx=FAR[2], pos=FAR[3], qw=FAR[4], kw_=FAR[5],
          eps=1e-5, inv=FAR[6], rot=128, style=0, Q=FAR[7], K=FAR[8], V=FAR[9], ws=FAR[10], ws_bytes=256):
    d = dims or _d()
    return lib.tb_norm_rope_append(ctypes.byref(d), qkv, stride, qb, n, ctx, pos, qw, kw_, eps, inv, rot, style, Q, K, V,
                                   ws, ws_bytes, None)


def test_norm_rope_append_refuses(lib):
    for kw, name in BAD_DIMS:
        assert _rope(lib, _d(**kw), stride=1 << 20) == _status(name), kw
    for kw in (dict(qkv=0), dict(qkv=FAKE + 8), dict(stride=48 * 128 - 8), dict(stride=48 * 128 + 4), dict(qb=0),
               dict(n=-1), dict(ctx=0), dict(pos=FAKE + 2), dict(qw=FAKE + 8), dict(kw_=FAKE + 2), dict(eps=-1e-9),
               dict(eps=float("nan")), dict(inv=0), dict(inv=FAKE + 4), dict(rot=136), dict(rot=12), dict(rot=-8),
               dict(style=2), dict(Q=0), dict(K=0), dict(V=FAKE + 8), dict(ws=0), dict(Q=FAR[0] + 16)):
        assert _rope(lib, **kw) == _lib.TB_ERR_INVALID_ARG, kw
    assert _rope(lib, ws_bytes=255) == _lib.TB_ERR_WORKSPACE
    assert _rope(lib, n=0x7fffffff) == _lib.TB_ERR_UNSUPPORTED
    assert _rope(lib, n=0, qkv=0, Q=0) == _lib.TB_OK


def _accept(lib, dims=None, layers=2, caches=FAR[0], qb=FAR[1], ctx=FAR[2], path=FAR[3], cap=8, plen=FAR[4],
            new=FAR[5], ws=FAR[6], ws_bytes=256):
    d = dims or _d()
    return lib.tb_tree_accept(ctypes.byref(d), layers, caches, qb, ctx, path, cap, plen, new, ws, ws_bytes, None)


def test_tree_accept_refuses(lib):
    for kw, name in BAD_DIMS:
        assert _accept(lib, _d(**kw)) == _status(name), kw
    for kw in (dict(layers=0), dict(caches=0), dict(caches=FAKE + 4), dict(qb=0), dict(ctx=FAKE + 1), dict(path=0),
               dict(plen=0), dict(new=0), dict(new=FAR[2]), dict(new=FAR[3] + 4), dict(new=FAR[4] + 4), dict(ws=0)):
        assert _accept(lib, **kw) == _lib.TB_ERR_INVALID_ARG, kw
    assert _accept(lib, cap=0) == _lib.TB_ERR_UNSUPPORTED and _accept(lib, cap=1025) == _lib.TB_ERR_UNSUPPORTED
    assert _accept(lib, ws_bytes=255) == _lib.TB_ERR_WORKSPACE


def test_binding_refuses_host_tensors(lib):
    d = _d(ctx_cap=64)
    kv = torch.zeros(2, 8, 64, 128, dtype=torch.bfloat16)
    Q = torch.zeros(4, 32, 128, dtype=torch.bfloat16)
    qb, ctx = torch.tensor([0, 2, 4], dtype=torch.int32), torch.tensor([2, 2], dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: _lib.prompt_attn(d, Q, kv, kv, qb, 2, ctx, 0.1, Q, ws),
                 lambda: _lib.tree_attn(d, Q, kv, kv, qb, 2, ctx, torch.zeros(4, 1, dtype=torch.int32), 0.1, Q, ws),
                 lambda: _lib.norm_rope_append(d, torch.zeros(4, 48 * 128, dtype=torch.bfloat16), qb, ctx, None, None,
                                               None, 0.0, None, False, Q, kv, kv, ws),
                 lambda: _lib.tree_accept(d, 1, torch.zeros(2, dtype=torch.int64), qb, ctx,
                                          torch.zeros(2, 4, dtype=torch.int32), ctx, ctx, ws)):
        with pytest.raises(_lib.TbError, match="device tensors"):
            call()
