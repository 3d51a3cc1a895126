"""Prompt and tree attention where the work is dealt out in equal shares of all
tiles, at shapes named by what they reach in that rule (tests/multi_dealing.py
restates it), against the 64-bit reference and tolerance of test_gpu_multi."""
import math

import numpy as np
import pytest
import torch

import query_aware_sparse_tb_b200 as tb
import test_gpu_multi as multi
from multi_dealing import Dealing
from query_aware_sparse_tb_b200 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


def fill_shared_memory():
    """A matrix product whose operand tiles stay behind in the SMs' shared memory."""
    a = torch.full((2048, 2048), 3.0, dtype=torch.bfloat16, device=DEV)
    return a @ a


def run(n, T, hkv, G, d, tree, cap=None, seed=0, repeats=1, before=None, flags=0):
    hq = hkv * G
    g = torch.Generator(device=DEV).manual_seed(seed)
    cap = cap or (max(T) + 127) // 128 * 128
    K, V = multi.make_cache(g, len(n), hkv, cap, d, T)
    total = sum(n)
    Q = torch.randn(total + 2, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    dm, mx = tb.dims(len(n), hq, hkv, d, 16, cap), max(n)
    scale = 1 / math.sqrt(d)
    size = (tb.tree_attn_workspace_bytes if tree else tb.prompt_attn_workspace_bytes)(dm, total + 2, mx)
    assert size > 1 << 20, "whole items, not shares"
    ws, qb, ctx = tb.workspace(size), multi.i32(multi.starts(n)), multi.i32(T)
    masks = mask = None
    if tree:
        r = np.random.RandomState(seed)
        masks = [multi.random_tree(k, r) for k in n]
        words = (mx + 31) // 32
        mask = torch.cat([multi.pack_rows([row for m in masks for row in m], words),
                          torch.zeros(2, words, dtype=torch.int32, device=DEV)])
    outs = []
    for _ in range(repeats):
        out = torch.full((total + 2, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
        if before:
            before()
        if tree:
            tb.tree_attn(dm, Q, K, V, qb, mx, ctx, mask, scale, out, ws)
        else:
            tb.prompt_attn(dm, Q, K, V, qb, mx, ctx, scale, out, ws)
        assert tb.workspace_check(ws) == flags
        assert (out[total:] == 7).all()
        outs.append(out[:total])
    assert all(torch.equal(o, outs[0]) for o in outs)
    see = multi.tree_see(masks, n, T) if tree else multi.causal(n, T)
    ref, tol = multi.reference(Q[:total], K, V, n, T, scale, see)
    multi.check(outs[0], ref, tol, f"{n} {T}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,T,hkv,G", [
    ([200], [3225], 32, 1),
    ([200], [3250], 32, 1),
    ([300] * 4, [4300] * 4, 8, 4),
    ([300] * 4, [9400] * 4, 8, 4),
])
def test_a_share_that_begins_behind_the_first_slots_tokens(n, T, hkv, G, d):
    """A CTA's first segment of two row blocks may hold only tiles that the
    first block does not see; whatever shared memory held before must not
    matter to it."""
    assert Dealing(n, T, hkv, G, False).check().slot0_without_tiles() > 0
    run(n, T, hkv, G, d, False, cap=12288, seed=3, repeats=3, before=fill_shared_memory)


def test_a_q_begin_that_does_not_rise_stays_in_the_join_list():
    """Overlapping sequences are more items than the host's bound.  Entries past
    the list of join entries would begin to overwrite state 0, which no CTA
    writes (nothing begins before the first share)."""
    B, tokens, d, cap, sms = 100, 300, 64, 16384, torch.cuda.get_device_properties(0).multi_processor_count
    with pytest.raises(AssertionError, match="list not written whole"):
        Dealing([tokens, 0] * (B // 2), [600] * B, 1, 4, False, n_tokens=tokens, ctas=sms).check()
    g = torch.Generator(device=DEV).manual_seed(1)
    K, V = multi.make_cache(g, B, 1, cap, d, [600] * B)
    Q = torch.randn(tokens, 4, d, generator=g, device=DEV).to(torch.bfloat16)
    out, dm = torch.zeros_like(Q), tb.dims(B, 4, 1, d, 16, cap)
    ws = tb.workspace(tb.prompt_attn_workspace_bytes(dm, tokens, tokens))
    assert ws.numel() > 1 << 20
    ws[256:] = 0xA5
    tb.prompt_attn(dm, Q, K, V, multi.i32([0, tokens] * (B // 2) + [0]), tokens, multi.i32([600] * B), 0.125, out, ws)
    torch.cuda.synchronize()
    states = 2 * sms * (d + 2) * 256 * 4
    assert (ws[-states:][:(d + 2) * 256 * 4] == 0xA5).all()


def test_decode_attention_takes_turns_on_the_workspace():
    """Verification and the decode step behind it on one workspace: the states
    of the shares must not lie where the decode attention keeps its tickets."""
    B, hkv, d, cap = 3, 2, 128, 8192
    n, T = [20, 9, 1], [5000, 3000, 7000]
    g = torch.Generator(device=DEV).manual_seed(4)
    K, V = multi.make_cache(g, B, hkv, cap, d, T)
    dm, scale = tb.dims(B, 4 * hkv, hkv, d, 16, cap), 1 / math.sqrt(d)
    Q = torch.randn(30, 4 * hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    last = Q[[19, 28, 29]].contiguous()
    r = np.random.RandomState(4)
    mask = multi.pack_rows([row for k in n for row in multi.random_tree(k, r)], 1)
    qb, ctx = multi.i32(multi.starts(n)), multi.i32(T)
    sizes = [tb.tree_attn_workspace_bytes(dm, 30, 20), tb.prompt_attn_workspace_bytes(dm, 30, 20),
             tb.attn_workspace_bytes(dm)]
    assert min(sizes[:2]) > 1 << 20

    def tree(ws):
        out = torch.zeros_like(Q)
        tb.tree_attn(dm, Q, K, V, qb, 20, ctx, mask, scale, out, ws)
        return out

    def prompt(ws):
        out = torch.zeros_like(Q)
        tb.prompt_attn(dm, Q, K, V, qb, 20, ctx, scale, out, ws)
        return out

    def decode(ws):
        out = torch.zeros(B, 4 * hkv, d, device=DEV)
        tb.decode_attn(dm, last, K, V, ctx, scale, out, ws)
        return out

    calls = [tree, prompt, decode]
    want = [f(tb.workspace(size)) for f, size in zip(calls, sizes)]
    shared = tb.workspace(max(sizes))
    for k in (0, 2, 1, 2, 2, 0, 1, 2):
        assert torch.equal(calls[k](shared), want[k]), calls[k].__name__
    assert tb.workspace_check(shared) == 0


def ragged(sizes, B, lo, hi, seed):
    r = np.random.RandomState(seed)
    n = [int(x) for x in r.choice(sizes, B)]
    return n, [k + int(x) for k, x in zip(n, r.randint(lo, hi, B))]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("n,T,hkv,d,cap", [
    (*ragged([0, 1, 3, 26, 33, 60, 70], 40, 2000, 8000, 7), 8, 64, 8192),   # 312 items, sequences without tokens among them
    (*ragged([100], 16, 12000, 16000, 8), 8, 128, 16384),                   # 256 items
    (*ragged([1, 26, 60, 64], 32, 4000, 15000, 9), 8, 64, 16384),
])
def test_shares_with_more_items_than_ctas(n, T, hkv, d, cap, tree):
    """The join entries are the CTAs', not the items'."""
    assert not Dealing(n, T, hkv, 4, tree, n_tokens=sum(n) + 2).check().by_item
    run(n, T, hkv, 4, d, tree, cap=cap, seed=5, repeats=2)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("hkv,d", [(1, 64), (1, 128), (4, 64)])
def test_shares_of_more_sequences_than_a_warp_looks_at_once(hkv, d, tree):
    """70 sequences: the line, its search and the report go on past 32; with one
    KV head the join entries are the items', with four the CTAs'."""
    n, T = ragged([0, 1, 3, 26, 33, 60], 70, 0, 8000, 7)
    assert Dealing(n, T, hkv, 4, tree, n_tokens=sum(n) + 2).check().by_item == (hkv == 1)
    run(n, T, hkv, 4, d, tree, cap=8192, seed=6, repeats=2)


@pytest.mark.parametrize("hkv", [1, 4])
def test_shares_with_tokens_that_have_no_row(hkv):
    """Sequences longer than their lengths among 40, in the second 32 too: their
    first tokens, whole items of them, see nothing and give 0."""
    n, T = ragged([0, 1, 26, 60], 40, 100, 8000, 11)
    for b, (k, t) in {3: (200, 100), 20: (30, 4), 35: (140, 9), 39: (65, 64)}.items():
        n[b], T[b] = k, t
    dealing = Dealing(n, T, hkv, 4, False, n_tokens=sum(n) + 2).check()
    assert any(tiles == 0 for _, _, _, tiles, _, _ in dealing.line) and dealing.by_item == (hkv == 1)
    run(n, T, hkv, 4, 64, False, cap=8192, seed=8, flags=_lib.TB_FLAG_CTX_RANGE)


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite_where_the_first_slot_has_no_tile(d):
    """The list of V rows taken out is written while a slot without tiles ends."""
    n, T, hkv = [200], [3225], 32
    assert Dealing(n, T, hkv, 1, False).slot0_without_tiles() > 0
    g = torch.Generator(device=DEV).manual_seed(13)
    K, V = multi.make_cache(g, 1, hkv, 12288, d, T)
    clean = V.clone()
    for row, value in ((T[0] - 1, float("nan")), (T[0] - 40, float("inf")), (T[0] - 190, float("nan"))):
        V[:, :, row, 7], clean[:, :, row, 7] = value, 0
    Q = torch.randn(200, hkv, d, generator=g, device=DEV).to(torch.bfloat16)
    dm, scale = tb.dims(1, hkv, hkv, d, 16, 12288), 1 / math.sqrt(d)
    ws = tb.workspace(tb.prompt_attn_workspace_bytes(dm, 200, 200))
    assert ws.numel() > 1 << 20
    ref, tol = multi.reference(Q, K, clean, n, T, scale, multi.causal(n, T))
    keep = [c for c in range(d) if c != 7]
    for _ in range(3):
        fill_shared_memory()
        out = torch.zeros_like(Q)
        tb.prompt_attn(dm, Q, K, V, multi.i32([0, 200]), 200, multi.i32(T), scale, out, ws)
        assert tb.workspace_check(ws) == 0
        assert out[10:, :, 7].isnan().all()                # tokens from the first NaN's row on
        multi.check(out[:10], ref[:10], tol[:10], "tokens before")
        multi.check(out[10:, :, keep], ref[10:, :, keep], tol[10:, :, keep], "other values")


@pytest.mark.parametrize("tree", [False, True])
def test_short_sequences_in_a_large_cache(tree):
    """The rule goes by the capacity: sequences of one to three tiles are shared
    out too, to few CTAs."""
    n, _ = ragged(range(1, 301), 16, 0, 1, 3)
    T = [k + (j % 3) * 10 for j, k in enumerate(n)]
    dealing = Dealing(n, T, 2, 4, tree, n_tokens=sum(n) + 2).check()
    assert dealing.shares < 148
    run(n, T, 2, 4, 64, tree, cap=65536, seed=9, repeats=2)


@pytest.mark.parametrize("cap", [1152, 32768])        # whole items; shares
@pytest.mark.parametrize("d,G", [(64, 4), (128, 16)])
def test_the_largest_tree_with_odd_rows_in_every_tile(d, G, cap):
    """1,024 drafted tokens that begin and end inside a tile: nine tiles with
    values that are not finite, each seen by its own token and one other."""
    n, T, hkv = [1024], [1061], 2
    g = torch.Generator(device=DEV).manual_seed(d)
    K, V = multi.make_cache(g, 1, hkv, cap, d, T)
    clean = V.clone()
    r = np.random.RandomState(d)
    mask = r.rand(1024, 1024) < 0.02
    odd = list(range(3, 1024, 120))
    mask[:, odd] = False
    seen = set()
    for k, j in enumerate(odd):
        other = (j * 7 + 500) % 1024
        mask[j, j] = mask[other, j] = True
        seen |= {j, other}
        V[:, :, 37 + j, 7], clean[:, :, 37 + j, 7] = float("nan") if k % 2 else float("inf"), 0
    Q = torch.randn(1024, hkv * G, d, generator=g, device=DEV).to(torch.bfloat16)
    out, dm, scale = torch.zeros_like(Q), tb.dims(1, hkv * G, hkv, d, 16, cap), 1 / math.sqrt(d)
    ws = tb.workspace(tb.tree_attn_workspace_bytes(dm, 1024, 1024))
    assert (ws.numel() > 256) == (cap > 2000)
    tb.tree_attn(dm, Q, K, V, multi.i32([0, 1024]), 1024, multi.i32(T), multi.pack_rows(mask, 32), scale, out, ws)
    assert tb.workspace_check(ws) == 0
    ref, tol = multi.reference(Q, K, clean, n, T, scale, multi.tree_see([mask], n, T))
    dirty = torch.zeros(1024, dtype=torch.bool, device=DEV)
    dirty[sorted(seen)] = True
    assert not out[dirty][:, :, 7].isfinite().any()
    multi.check(out[~dirty], ref[~dirty], tol[~dirty], "tokens that see none")
    keep = [c for c in range(d) if c != 7]
    multi.check(out[:, :, keep], ref[:, :, keep], tol[:, :, keep], "other values")


def test_calls_from_several_host_threads():
    """Each thread its stream, workspace and outputs; the cache is shared."""
    import threading
    n, T, hkv, d = [40, 9], [3000, 700], 2, 128
    g = torch.Generator(device=DEV).manual_seed(1)
    K, V = multi.make_cache(g, 2, hkv, 4096, d, T)
    Q = torch.randn(49, 8, d, generator=g, device=DEV).to(torch.bfloat16)
    dm, scale, qb, ctx = tb.dims(2, 8, hkv, d, 16, 4096), 1 / math.sqrt(d), multi.i32([0, 40, 49]), multi.i32(T)
    size = tb.prompt_attn_workspace_bytes(dm, 49, 40)
    want = torch.zeros_like(Q)
    tb.prompt_attn(dm, Q, K, V, qb, 40, ctx, scale, want, tb.workspace(size))
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ws = tb.workspace(size)
                for _ in range(50):
                    out = torch.zeros_like(Q)
                    tb.prompt_attn(dm, Q, K, V, qb, 40, ctx, scale, out, ws)
                    with pytest.raises(tb.TbError, match="max_new"):
                        tb.prompt_attn(dm, Q, K, V, qb, 0, ctx, scale, out, ws)
                    stream.synchronize()
                    if not torch.equal(out, want):
                        wrong.append("differs")
                if tb.workspace_check(ws):
                    wrong.append("flag")
        except BaseException as e:  # noqa: BLE001
            wrong.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]
