"""Calls for several new tokens that the documentation allows and that are easy
to get wrong."""
import math

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


# ------------------------------------------------------------------ into the decode path

@pytest.mark.parametrize("d", [64, 128])
def test_a_prompt_leads_into_the_sparse_decode_step(d):
    """A prompt fills the cache, its keys are projected, the next token is
    scored, selects and attends: captured without a wait between the calls and
    replayed over cleared caches, the same bits as with a wait after each call.
    With a budget of the whole context the step is dense attention."""
    hq, hkv, dp, cap, n, T = 8, 2, 16, 640, [300, 41], [300, 41]
    sink, window, nbr = 4, 8, 1
    dm, total, scale = tb.dims(2, hq, hkv, d, dp, cap), sum(n), 1 / math.sqrt(d)
    g = torch.Generator(device=DEV).manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    qkv, step_qkv = rnd(total, (hq + 2 * hkv) * d), rnd(2, (hq + 2 * hkv) * d)
    Wk, qp = rnd(hkv, dp, d), torch.randn(2, hq, dp, generator=g, device=DEV)
    inv = 10000.0 ** (-2 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)
    qb, one, ctx, ctx1 = i32(multi.starts(n)), i32([0, 1, 2]), i32(T), i32([t + 1 for t in T])
    begin, count = i32([0, 0]), i32([t + 1 for t in T])

    def buffers(budget):
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
        return dict(K=z(2, hkv, cap, d), V=z(2, hkv, cap, d), Kp=z(2, hkv, cap, dp), Q=z(total, hq, d), Q1=z(2, hq, d),
                    out=z(total, hq, d), out1=z(2, hq, d, t=torch.float32), budget=budget,
                    idx=z(2, hq, min(3 * budget, cap), t=torch.int32), cnt=z(2, hq, t=torch.int32),
                    bits=z(2, hq, cap // 32, t=torch.int32), ws=tb.workspace(256),
                    wp=tb.workspace(tb.prompt_attn_workspace_bytes(dm, total, 300)),
                    wsel=tb.workspace(tb.score_select_workspace_bytes(dm)), wa=tb.workspace(tb.attn_workspace_bytes(dm)))

    def chain(y, after=lambda: None):
        rope = lambda x, q, c, Q: tb.norm_rope_append(dm, x, q, c, None, None, None, 0.0, inv, False, Q, y["K"], y["V"], y["ws"])  # noqa: E731
        for call in (
            lambda: rope(qkv, qb, ctx, y["Q"]),
            lambda: tb.prompt_attn(dm, y["Q"], y["K"], y["V"], qb, 300, ctx, scale, y["out"], y["wp"]),
            lambda: rope(step_qkv, one, ctx1, y["Q1"]),
            lambda: tb.project_keys(dm, y["K"], Wk, y["Kp"], begin, count, 301, y["ws"]),
            lambda: tb.score_select(dm, qp, hq * dp, y["Kp"], ctx1, sink, window, y["budget"], nbr, y["idx"], y["cnt"],
                                    y["bits"], y["wsel"]),
            lambda: tb.sparse_decode_attn(dm, y["Q1"], y["K"], y["V"], ctx1, sink, window, y["bits"], scale, y["out1"],
                                          y["wa"]),
        ):
            call()
            after()

    for budget in (16, cap):
        want, got = buffers(budget), buffers(budget)
        chain(want, torch.cuda.synchronize)
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                chain(got)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(3):
            for name in ("K", "V", "Kp", "Q", "Q1", "out", "out1", "bits"):
                got[name].zero_()
            graph.replay()
            torch.cuda.synchronize()
            for name in ("K", "V", "Kp", "Q", "Q1", "out", "out1", "bits", "cnt"):
                assert torch.equal(got[name], want[name]), (budget, name)
        for name in ("ws", "wp", "wsel", "wa"):
            assert tb.workspace_check(got[name]) == 0 and tb.workspace_check(want[name]) == 0
        multi.check(want["out"], *multi.reference(want["Q"], want["K"], want["V"], n, T, scale, multi.causal(n, T)), "prompt")
    T1 = [t + 1 for t in T]
    multi.check(want["out1"], *multi.reference(want["Q1"], want["K"], want["V"], [1, 1], T1, scale, multi.causal([1, 1], T1)),
                "decode step")


# ------------------------------------------------------------------ nothing beside the outputs

def guarded(shape, dtype, fill, pad=4096):
    """A tensor in the middle of a buffer of a known pattern, and a check that
    the pattern beside it is still there."""
    nbytes = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((pad + nbytes + pad,), 0x5C, dtype=torch.uint8, device=DEV)
    t = buf[pad:pad + nbytes].view(dtype).view(shape)
    if fill is not None:
        t.copy_(fill)
    return t, lambda: bool((buf[:pad] == 0x5C).all()) and bool((buf[pad + nbytes:] == 0x5C).all())


@pytest.mark.parametrize("cap", [513, 32768])         # whole items; shares
@pytest.mark.parametrize("d", [64, 128])
def test_calls_write_nothing_beside_their_outputs(d, cap):
    n, T, hq, hkv = [33, 0, 70, 1], [400, 0, 513, 1], 8, 2
    g = torch.Generator(device=DEV).manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    dm, total = tb.dims(4, hq, hkv, d, 16, cap), sum(n)
    qb, ctx = i32(multi.starts(n)), i32(T)
    K, k_ok = guarded((4, hkv, cap, d), torch.bfloat16, rnd(4, hkv, cap, d))
    V, v_ok = guarded((4, hkv, cap, d), torch.bfloat16, rnd(4, hkv, cap, d))
    Q, q_ok = guarded((total, hq, d), torch.bfloat16, None)
    out, o_ok = guarded((total, hq, d), torch.bfloat16, None)
    new_len, l_ok = guarded((4,), torch.int32, None)
    small, s_ok = guarded((256,), torch.uint8, torch.zeros(256, dtype=torch.uint8, device=DEV))
    qkv = rnd(total, (hq + 2 * hkv) * d)
    tb.norm_rope_append(dm, qkv, qb, ctx, None, None, None, 0.0, None, False, Q, K, V, small)
    x = qkv.view(total, hq + 2 * hkv, d)
    assert torch.equal(Q, x[:, :hq]) and q_ok() and k_ok() and v_ok() and s_ok()
    K0, V0 = K.clone(), V.clone()
    for tree in (False, True):
        size = (tb.tree_attn_workspace_bytes if tree else tb.prompt_attn_workspace_bytes)(dm, total, 70)
        assert (size > 256) == (cap > 1000)
        ws, w_ok = guarded((size,), torch.uint8, torch.zeros(size, dtype=torch.uint8, device=DEV))
        for _ in range(2):
            if tree:
                mask = torch.full((total, 3), -1, dtype=torch.int32, device=DEV)
                tb.tree_attn(dm, Q, K, V, qb, 70, ctx, mask, 0.1, out, ws)
            else:
                tb.prompt_attn(dm, Q, K, V, qb, 70, ctx, 0.1, out, ws)
        assert tb.workspace_check(ws) == 0 and w_ok() and o_ok() and q_ok() and k_ok() and v_ok()
        assert torch.equal(K, K0) and torch.equal(V, V0) and torch.equal(Q, x[:, :hq])
    caches = torch.tensor([K.data_ptr(), V.data_ptr()], dtype=torch.int64, device=DEV)
    path = i32([list(range(1, 33)), [0] * 32, list(range(38, 70)), [0] * 32])
    tb.tree_accept(dm, 1, caches, qb, ctx, path, i32([32, 0, 32, 1]), new_len, small)
    assert tb.workspace_check(small) == 0 and new_len.tolist() == [399, 0, 475, 1]
    for now, was in ((K, K0), (V, V0)):
        want = was.clone()
        want[0, :, 367:399] = was[0, :, 368:400]
        want[2, :, 443:475] = was[2, :, 481:513]
        assert torch.equal(now, want)
    assert k_ok() and v_ok() and l_ok() and s_ok()
