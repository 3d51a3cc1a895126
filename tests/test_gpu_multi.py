"""The calls that take several new tokens of a sequence at once, against 64-bit
references of their formulas: norms + rotation + cache write, prompt
attention, tree attention and tree acceptance, and a run of them together
with the decode step that follows.

Tolerances are the arithmetic's.  u = 2^-8 is a bf16 rounding's largest
relative error, e = 2^-24 an fp32 one's.

  attention  |out - ref| <= u |ref| + A (u + 2 w + 2 e N) with A = sum p|v| /
             sum p, N the row's number of terms and w the largest error of a
             weight's exponent: the fp32 dot product (d e sum|q k| scale), the
             product and difference in log2 units (4 e (|l| + 8)) and the
             exponential (2^-21); twice, for numerator and denominator.  The
             u in the brackets is the weights' rounding before the product
             with V.
  rotation   |y - ref| <= u |ref| + 24 e (|a| + |b|) for a pair (a, b): about
             ten fp32 operations on each value, and an angle whose fp32
             rounding is at most 2^-24 of half a turn (pi e)."""
import math

import numpy as np
import pytest
import torch

import query_aware_sparse_tb_b200 as tb
from query_aware_sparse_tb_b200 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, E = 2.0 ** -8, 2.0 ** -24
F64 = torch.float64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def make_cache(g, B, hkv, cap, d, T, heavy=True):
    """K and V with NaN in every row at and past the length."""
    K = torch.randn(B, hkv, cap, d, generator=g, device=DEV).to(torch.bfloat16)
    V = torch.randn(B, hkv, cap, d, generator=g, device=DEV).to(torch.bfloat16)
    if heavy:
        K = torch.where(torch.rand(B, hkv, cap, 1, generator=g, device=DEV) < 0.02, K * 4, K)
    for b, t in enumerate(T):
        K[b, :, t:] = float("nan")
        V[b, :, t:] = float("nan")
    return K, V


def reference(Q, K, V, n, T, scale, see):
    """(ref, tolerance) [tokens][Hq][d] in float64.  see(b, i0, i1): bool
    [i1 - i0][T] of the rows tokens i0 .. i1 - 1 of sequence b attend to."""
    hq, d, hkv = Q.shape[1], Q.shape[2], K.shape[1]
    G = hq // hkv
    ref = torch.zeros(Q.shape, dtype=F64, device=DEV)
    tol = torch.zeros_like(ref)
    s = starts(n)
    for b in range(len(n)):
        if n[b] == 0:
            continue
        for i0 in range(0, n[b], 512):
            i1 = min(n[b], i0 + 512)
            ok = see(b, i0, i1)
            for h in range(hq):
                q = Q[s[b] + i0:s[b] + i1, h].to(F64)
                k, v = K[b, h // G, :T[b]].to(F64), V[b, h // G, :T[b]].to(F64)
                l = (q @ k.T) * scale
                mag = (q.abs() @ k.abs().T) * scale
                l = l.masked_fill(~ok, -math.inf)
                top = l.amax(1, keepdim=True)
                dead = torch.isinf(top)
                p = torch.where(dead, 0.0, torch.exp(l - torch.where(dead, 0.0, top)))
                den = p.sum(1, keepdim=True)
                den = torch.where(dead, 1.0, den)
                o = (p @ v) / den
                A = (p @ v.abs()) / den
                w = d * E * mag.masked_fill(~ok, 0).amax(1) + 4 * E * (l.masked_fill(~ok, 0).abs().amax(1) * 1.45 + 8) + 2.0 ** -21
                N = ok.sum(1)
                ref[s[b] + i0:s[b] + i1, h] = o
                tol[s[b] + i0:s[b] + i1, h] = U * o.abs() + A * (U + 2 * w + 2 * E * N)[:, None]
    return ref, tol


def causal(n, T):
    def see(b, i0, i1):
        t = torch.arange(T[b], device=DEV)
        return t[None] <= (T[b] - n[b] + torch.arange(i0, i1, device=DEV))[:, None]
    return see


def check(out, ref, tol, what=""):
    err = (out.to(F64) - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((err / tol).nan_to_num(1e9).max()):.3g} x the tolerance"


def run_prompt(n, T, hq, hkv, d, cap=None, seed=0, max_new=None, extra=3, scale=None, stream=None, K=None, V=None,
               Q=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B = len(n)
    cap = cap or (max(T) + 127) // 128 * 128
    if K is None:
        K, V = make_cache(g, B, hkv, cap, d, T)
    total = sum(n)
    if Q is None:
        Q = torch.randn(total + extra, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.full((total + extra, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    dm = tb.dims(B, hq, hkv, d, 16, cap)
    mn = max_new or max(n)
    ws = tb.workspace(tb.prompt_attn_workspace_bytes(dm, total + extra, mn))
    scale = scale or 1 / math.sqrt(d)
    tb.prompt_attn(dm, Q, K, V, i32(starts(n)), mn, i32(T), scale, out, ws)
    torch.cuda.synchronize()
    assert tb.workspace_check(ws) == 0
    assert (out[total:] == 7).all()  # behind the last sequence
    return Q, K, V, out, scale


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,T", [
    ([1], [1]),                         # one token, nothing before it
    ([5], [5]),
    ([33], [33]),                       # one token in the second slot
    ([64], [64]),
    ([65], [65]),                       # two items
    ([129], [129]),
    ([300], [300]),
    ([1, 0, 7, 31, 32, 100], [1, 0, 7, 31, 32, 100]),
])
def test_prompt_whole(n, T, d):
    Q, K, V, out, scale = run_prompt(n, T, 8, 2, d)
    ref, tol = reference(Q, K, V, n, T, scale, causal(n, T))
    check(out[:sum(n)], ref[:sum(n)], tol[:sum(n)], f"{n}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,T", [
    ([1, 1, 1], [1, 700, 1025]),        # decode steps
    ([3, 40, 64, 100], [128, 129, 1000, 357]),
    ([200, 0, 17], [1201, 50, 4017]),
    ([96], [5000]),
])
def test_prompt_chunks_behind_cached_rows(n, T, d):
    Q, K, V, out, scale = run_prompt(n, T, 8, 2, d, seed=1)
    ref, tol = reference(Q, K, V, n, T, scale, causal(n, T))
    check(out[:sum(n)], ref[:sum(n)], tol[:sum(n)], f"{n}")


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_prompt_group_sizes(G):
    n, T = [70, 1, 150], [90, 300, 150]
    Q, K, V, out, scale = run_prompt(n, T, 3 * G, 3, 128, seed=2)
    ref, tol = reference(Q, K, V, n, T, scale, causal(n, T))
    check(out[:sum(n)], ref[:sum(n)], tol[:sum(n)], f"G={G}")


@pytest.mark.parametrize("cap,T", [(1, 1), (2, 2), (5, 4), (127, 127), (129, 129)])
def test_caches_smaller_than_a_tile_and_of_odd_size(cap, T):
    for n in (1, T):
        Q, K, V, out, scale = run_prompt([n], [T], 1, 1, 64, seed=cap, cap=cap)
        ref, tol = reference(Q, K, V, [n], [T], scale, causal([n], [T]))
        check(out[:n], ref[:n], tol[:n], f"cap {cap}, n {n}")


def test_prompt_long_covers_every_wave():
    n, T = [2500, 700], [2500, 1300]
    Q, K, V, out, scale = run_prompt(n, T, 32, 8, 128, seed=3)
    ref, tol = reference(Q, K, V, n, T, scale, causal(n, T))
    check(out[:sum(n)], ref[:sum(n)], tol[:sum(n)])


# ------------------------------------------------------------------ trees

def random_tree(n, r):
    """Rows of bools [n][n]: ancestors and self of a random tree whose parents
    come before their children."""
    m = np.zeros((n, n), dtype=bool)
    for i in range(n):
        p = int(r.randint(-1, i))
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def pack_rows(rows, words):
    out = np.zeros((len(rows), words), dtype=np.uint32)
    for i, row in enumerate(rows):
        for j in np.flatnonzero(row):
            out[i, j // 32] |= np.uint32(1 << (int(j) % 32))
    return torch.tensor(out.view(np.int32), device=DEV)


def tree_see(masks, n, T):
    def see(b, i0, i1):
        ok = torch.ones(i1 - i0, T[b], dtype=torch.bool, device=DEV)
        ok[:, T[b] - n[b]:] = torch.tensor(masks[b][i0:i1], device=DEV)
        return ok
    return see


def run_tree(n, T, masks, hq, hkv, d, max_new=None, seed=0, extra=2, cap=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cap = cap or (max(T) + 63) // 64 * 64
    K, V = make_cache(g, len(n), hkv, cap, d, T)
    total = sum(n)
    mn = max_new or max(n)
    words = (mn + 31) // 32
    Q = torch.randn(total + extra, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    mask = torch.cat([pack_rows([row for m in masks for row in m], words),
                      torch.full((extra, words), -1, dtype=torch.int32, device=DEV)])
    out = torch.full((total + extra, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    dm = tb.dims(len(n), hq, hkv, d, 16, cap)
    ws = tb.workspace(tb.tree_attn_workspace_bytes(dm, total + extra, mn))
    scale = 1 / math.sqrt(d)
    tb.tree_attn(dm, Q, K, V, i32(starts(n)), mn, i32(T), mask, scale, out, ws)
    torch.cuda.synchronize()
    assert tb.workspace_check(ws) == 0
    assert (out[total:] == 7).all()
    return Q, K, V, out, scale


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,T", [
    ([1], [1]),
    ([1, 4, 0, 26], [3, 4, 900, 5000]),       # a tree with nothing before it among them
    ([32, 33, 64], [160, 161, 2000]),         # drafted rows that begin and end inside a tile
    ([65, 100, 128], [129, 1100, 300]),       # several items per sequence
    ([300], [700]),                           # the drafted rows span several tiles
])
def test_tree(n, T, d):
    r = np.random.RandomState(5)
    masks = [random_tree(k, r) for k in n]
    Q, K, V, out, scale = run_tree(n, T, masks, 8, 2, d)
    ref, tol = reference(Q, K, V, n, T, scale, tree_see(masks, n, T))
    check(out[:sum(n)], ref[:sum(n)], tol[:sum(n)], f"{n}")


@pytest.mark.parametrize("G", [1, 2, 8, 16])
def test_tree_group_sizes(G):
    n, T = [33, 1, 20], [600, 40, 20]
    r = np.random.RandomState(G)
    masks = [random_tree(k, r) for k in n]
    Q, K, V, out, scale = run_tree(n, T, masks, 2 * G, 2, 64, seed=G)
    ref, tol = reference(Q, K, V, n, T, scale, tree_see(masks, n, T))
    check(out[:54], ref[:54], tol[:54], f"G={G}")


def test_tree_any_mask_and_rows_that_see_nothing():
    """Masks that are no trees (later tokens, no self), with and without rows
    before the drafted ones; a token that sees nothing gets 0."""
    n, T = [40, 40, 7], [40, 300, 7]
    r = np.random.RandomState(6)
    masks = [r.rand(k, k) < 0.3 for k in n]
    masks[0][3] = False
    masks[0][39] = False
    masks[1][5] = False
    masks[2][:] = False
    Q, K, V, out, scale = run_tree(n, T, masks, 16, 2, 128, max_new=77, seed=4)
    ref, tol = reference(Q, K, V, n, T, scale, tree_see(masks, n, T))
    check(out[:87], ref[:87], tol[:87])
    assert (out[3] == 0).all() and (out[39] == 0).all() and (out[80:87] == 0).all()


def test_chain_tree_equals_prompt_and_one_token_equals_decode():
    n, T = [1, 20, 33], [700, 515, 1033]
    masks = [np.tril(np.ones((k, k), dtype=bool)) for k in n]
    Q, K, V, out, scale = run_tree(n, T, masks, 8, 2, 128, seed=8)
    _, _, _, out2, _ = run_prompt(n, T, 8, 2, 128, extra=2, K=K, V=V, Q=Q, cap=K.shape[2])
    assert torch.equal(out, out2)
    # the decode entry point on the same cache: its result is fp32, this one's
    # bf16, and both weights and result are rounded here
    dm = tb.dims(3, 8, 2, 128, 16, K.shape[2])
    last = torch.tensor([0, 20, 53], device=DEV)
    dec = torch.zeros(3, 8, 128, device=DEV)
    ws = tb.workspace(tb.attn_workspace_bytes(dm))
    tb.decode_attn(dm, Q[last].contiguous(), K, V, i32(T), scale, dec, ws)
    ref, tol = reference(Q, K, V, n, T, scale, causal(n, T))
    check(dec, ref[last], tol[last], "decode")
    check(out[last], ref[last], tol[last], "tree")


# ------------------------------------------------------------------ norms, rotation, cache write

def rope_reference(x, w, eps, pos, inv_freq, interleaved):
    """(ref, tolerance) of rows x [n][heads][d] at positions pos [n]."""
    d, y = x.shape[-1], x.to(F64)
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w.to(F64)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    z, mag = y.clone(), y.abs()
    if rot:
        ang = pos.to(F64)[:, None] * inv_freq
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        ia = torch.arange(0, rot, 2, device=DEV) if interleaved else torch.arange(rot // 2, device=DEV)
        ib = ia + 1 if interleaved else ia + rot // 2
        a, b = y[..., ia], y[..., ib]
        z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return z, U * z.abs() + 24 * E * mag


@pytest.mark.parametrize("d,hq,hkv,rot,inter,qn,kn", [
    (128, 32, 8, 128, False, True, True),
    (64, 8, 2, 64, False, True, True),
    (64, 8, 2, 64, True, True, False),
    (128, 8, 2, 40, False, False, True),
    (128, 8, 1, 56, True, False, False),
    (64, 3, 3, 8, False, True, True),
    (64, 7, 7, 0, False, True, True),
])
@pytest.mark.parametrize("own_pos", [False, True])
def test_norm_rope_append(d, hq, hkv, rot, inter, qn, kn, own_pos):
    n, T = [1, 0, 9, 130], [1, 0, 70, 131]
    g = torch.Generator(device=DEV).manual_seed(d + hq + rot)
    cap, total, extra = 140, sum(n), 4
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    wide = rnd(total + extra, (hq + 2 * hkv) * d + 24)     # rows further apart than their width
    qkv = wide[:, :(hq + 2 * hkv) * d]
    K0, V0 = rnd(4, hkv, cap, d), rnd(4, hkv, cap, d)
    K, V = K0.clone(), V0.clone()
    Q = torch.full((total + extra, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    qw, kw = (1 + rnd(d) / 4 if qn else None), (1 + rnd(d) / 4 if kn else None)
    inv = 500000.0 ** (-2 * torch.arange(rot // 2, dtype=F64, device=DEV) / rot) if rot else None
    s = starts(n)
    rows = [T[b] - n[b] + i for b in range(4) for i in range(n[b])]
    # positions far out: an angle in fp32 would be off by up to 2^-4 here
    pos = torch.randint(0, 1 << 20, (total + extra,), generator=g, device=DEV, dtype=torch.int32) if own_pos else None
    dm = tb.dims(4, hq, hkv, d, 16, cap)
    ws = tb.workspace(256)
    tb.norm_rope_append(dm, qkv, i32(s), i32(T), pos, qw, kw, 1e-5, inv, inter, Q, K, V, ws)
    torch.cuda.synchronize()
    assert tb.workspace_check(ws) == 0
    assert (Q[total:] == 7).all()
    P = pos[:total] if own_pos else torch.tensor(rows, device=DEV)
    x = qkv[:total].reshape(total, hq + 2 * hkv, d)
    ref, tol = rope_reference(x[:, :hq], qw, 1e-5, P, inv, inter)
    check(Q[:total], ref, tol, "Q")
    ref, tol = rope_reference(x[:, hq:hq + hkv], kw, 1e-5, P, inv, inter)
    seq = torch.tensor([b for b in range(4) for _ in range(n[b])], device=DEV)
    rows = torch.tensor(rows, device=DEV)
    check(K[seq, :, rows], ref, tol, "K")
    assert torch.equal(V[seq, :, rows], x[:, hq + hkv:])
    K[seq, :, rows], V[seq, :, rows] = K0[seq, :, rows], V0[seq, :, rows]
    assert torch.equal(K, K0) and torch.equal(V, V0)      # no other row was written


def test_norm_rope_append_many_sequences_and_tokens():
    """More sequences than one round of the search sees, empty ones among
    them, and enough tokens for a warp per token."""
    r = np.random.RandomState(3)
    n = [int(x) for x in r.choice([0, 0, 1, 3, 9], 1500)]
    T = [k + int(r.randint(0, 12)) for k in n]
    d, hq, hkv, cap, total = 64, 4, 1, 24, sum(n)
    assert total > 148 * 16
    g = torch.Generator(device=DEV).manual_seed(1)
    qkv = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device=DEV).to(torch.bfloat16)
    K = torch.zeros(len(n), hkv, cap, d, dtype=torch.bfloat16, device=DEV)
    V, Q = torch.zeros_like(K), torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEV)
    inv = 10000.0 ** (-2 * torch.arange(d // 2, dtype=F64, device=DEV) / d)
    ws = tb.workspace(256)
    tb.norm_rope_append(tb.dims(len(n), hq, hkv, d, 16, cap), qkv, i32(starts(n)), i32(T), None, None, None, 0.0, inv,
                        False, Q, K, V, ws)
    assert tb.workspace_check(ws) == 0
    seq = torch.tensor(np.repeat(np.arange(len(n)), n), device=DEV)
    row = torch.tensor(np.concatenate([np.arange(T[b] - n[b], T[b]) for b in range(len(n))]), device=DEV)
    x = qkv.view(total, hq + 2 * hkv, d)
    check(Q, *rope_reference(x[:, :hq], None, 0.0, row, inv, False), "Q")
    check(K[seq, :, row], *rope_reference(x[:, hq:hq + hkv], None, 0.0, row, inv, False), "K")
    assert torch.equal(V[seq, :, row], x[:, hq + hkv:])
    assert int((V.abs().sum(-1) > 0).sum()) <= total


def test_zero_rows_and_extreme_values_through_the_norm():
    """A row of zeros stays zero (eps > 0); rows whose squares fit fp32 come out
    finite."""
    d, hq, hkv = 128, 4, 1
    qkv = torch.zeros(3, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device=DEV)
    qkv[1] = 1e17
    qkv[2] = 1e-12
    K = torch.zeros(3, hkv, 4, d, dtype=torch.bfloat16, device=DEV)
    V, Q = torch.zeros_like(K), torch.zeros(3, hq, d, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    ws = tb.workspace(256)
    tb.norm_rope_append(tb.dims(3, hq, hkv, d, 16, 4), qkv, i32([0, 1, 2, 3]), i32([1, 1, 1]), None, w, w, 1e-6, None,
                        False, Q, K, V, ws)
    x = qkv.view(3, hq + 2 * hkv, d)
    check(Q, *rope_reference(x[:, :hq], w, 1e-6, torch.zeros(3, device=DEV), None, False))
    assert (Q[0] == 0).all() and (Q[1] == 1).all()


# ------------------------------------------------------------------ acceptance

@pytest.mark.parametrize("d", [64, 128])
def test_tree_accept(d):
    r = np.random.RandomState(d)
    n = [1, 0, 26, 64, 40, 1000, 3]
    T = [5, 9, 26, 500, 300, 1000, 3]
    L, B, hkv, cap = 3, len(n), 3, 1024
    g = torch.Generator(device=DEV).manual_seed(d)
    kv = torch.randn(L, 2, B, hkv, cap, d, generator=g, device=DEV).to(torch.bfloat16)
    want = kv.clone()
    step = B * hkv * cap * d * 2
    caches = torch.tensor([kv.data_ptr() + i * step for i in range(2 * L)], dtype=torch.int64, device=DEV)
    lens = [1, 0, 7, 33, 40, 700, 0]
    cap_p = 700
    path = np.full((B, cap_p), -9, dtype=np.int32)
    for b in range(B):
        p = np.sort(r.choice(max(n[b], 1), lens[b], replace=False))
        path[b, :lens[b]] = p
        base = T[b] - n[b]
        want[:, :, b, :, base:base + lens[b]] = kv[:, :, b, :, base + torch.tensor(p, dtype=torch.long, device=DEV)]
    new_len = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    ws = tb.workspace(256)
    tb.tree_accept(tb.dims(B, hkv * 4, hkv, d, 16, cap), L, caches, i32(starts(n)), i32(T), i32(path), i32(lens),
                   new_len, ws)
    assert tb.workspace_check(ws) == 0
    assert new_len.tolist() == [T[b] - n[b] + lens[b] for b in range(B)]
    assert torch.equal(kv, want)


def test_tree_accept_skips_and_reports_a_bad_path():
    B, hkv, cap, d = 6, 1, 32, 64
    n, T = [5] * B, [10, 10, 10, 4, 40, 10]
    kv = torch.randn(1, 2, B, hkv, cap, d, device=DEV).to(torch.bfloat16)
    want = kv.clone()
    caches = torch.tensor([kv[0, 0].data_ptr(), kv[0, 1].data_ptr()], dtype=torch.int64, device=DEV)
    path = [[1, 1, 2], [0, 5, 6], [-1, 2, 3], [1, 2, 3], [1, 2, 3], [1, 3, 4]]
    new_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    ws = tb.workspace(256)
    tb.tree_accept(tb.dims(B, 4, 1, d, 16, cap), 1, caches, i32(starts(n)), i32(T), i32(path), i32([3] * B), new_len,
                   ws)
    assert tb.workspace_check(ws) == _lib.TB_FLAG_BAD_PATH
    assert new_len.tolist() == T[:5] + [8]                # only the last one is sound
    want[0, :, 5, :, 5:8] = want[0, :, 5, :, [6, 8, 9]]
    assert torch.equal(kv, want)


# ------------------------------------------------------------------ conditions only the device sees

def test_lengths_out_of_range_are_reported_and_stay_in_bounds():
    hq, hkv, d, cap = 4, 1, 64, 256
    n, T = [10, 300, 4], [4, 9999, 0]      # fewer rows than tokens; beyond the cache; no length at all
    g = torch.Generator(device=DEV).manual_seed(0)
    K = torch.randn(3, hkv, cap, d, generator=g, device=DEV).to(torch.bfloat16)
    V = torch.randn(3, hkv, cap, d, generator=g, device=DEV).to(torch.bfloat16)
    total = sum(n)
    Q = torch.randn(total, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    out = torch.full_like(Q, 7.0)
    dm = tb.dims(3, hq, hkv, d, 16, cap)
    ws = tb.workspace(tb.prompt_attn_workspace_bytes(dm, total, 300))
    tb.prompt_attn(dm, Q, K, V, i32(starts(n)), 300, i32(T), 0.125, out, ws)
    assert tb.workspace_check(ws) == _lib.TB_FLAG_CTX_RANGE
    assert (out[:6] == 0).all()            # tokens without a row
    see = lambda b, i0, i1: causal([10], [4])(b, i0, i1)  # noqa: E731
    ref, tol = reference(Q[:10], K[:1], V[:1], [10], [4], 0.125, see)
    check(out[:10], ref, tol)
    out.fill_(7.0)
    tb.prompt_attn(dm, Q, K, V, i32([0, 10, 20, 30]), 4, i32([100, 100, 100]), 0.125, out, ws)  # max_new too small
    assert tb.workspace_check(ws) == _lib.TB_FLAG_CTX_RANGE
    assert (out[4:10] == 7).all() and (out[14:20] == 7).all() and not (out[:4] == 7).any()
    # a q_begin that runs backwards or past the tokens
    out.fill_(7.0)
    tb.prompt_attn(dm, Q, K, V, i32([5, 2, 400, 380]), 300, i32([100, 256, 100]), 0.125, out, ws)
    tb.workspace_check(ws)
    assert (out[:2] == 7).all()
    inv = torch.ones(d // 2, dtype=F64, device=DEV)
    qkv = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device=DEV).to(torch.bfloat16)
    K2, V2, Q2 = K.clone(), V.clone(), torch.zeros_like(Q)
    tb.norm_rope_append(dm, qkv, i32(starts(n)), i32(T), None, None, None, 0.0, inv, False, Q2, K2, V2, ws)
    assert tb.workspace_check(ws) == _lib.TB_FLAG_CTX_RANGE
    assert not (Q2 == 0).all(-1).any()     # every query row is written
    assert torch.equal(K2[0, :, 4:], K[0, :, 4:]) and torch.equal(K2[1:], K[1:])
    assert torch.equal(V2[0, 0, :4], qkv[6:10, (hq + hkv) * d:])


def test_prompt_is_deterministic_and_replays_in_a_graph():
    n, T = [40, 1, 90], [3000, 2500, 90]
    Q, K, V, out, scale = run_prompt(n, T, 8, 2, 128, seed=9, extra=0)
    dm = tb.dims(3, 8, 2, 128, 16, K.shape[2])
    ws = tb.workspace(tb.prompt_attn_workspace_bytes(dm, sum(n), 90))
    qb, ct, got = i32(starts(n)), i32(T), torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tb.prompt_attn(dm, Q, K, V, qb, 90, ct, scale, got, ws)
        with torch.cuda.graph(graph, stream=side):
            tb.prompt_attn(dm, Q, K, V, qb, 90, ct, scale, got, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    for k in range(3):                     # new values in the captured buffers
        Q.copy_(torch.randn_like(Q))
        want = torch.zeros_like(out)
        tb.prompt_attn(dm, Q, K, V, qb, 90, ct, scale, want, ws)
        torch.cuda.synchronize()
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert tb.workspace_check(ws) == 0


@pytest.mark.parametrize("d,hkv,cap", [(128, 2, 4096), (64, 8, 512)])  # equal shares of the tiles; whole items
def test_a_captured_drafting_step_follows_lengths_and_masks(d, hkv, cap):
    """Norm + rotation, tree attention and acceptance captured once, replayed
    with other sequence starts, lengths, positions, masks and paths."""
    B, hq, tokens, mn = 8, 4 * hkv, 120, 40
    dm = tb.dims(B, hq, hkv, d, 16, cap)
    g = torch.Generator(device=DEV).manual_seed(d)
    first = torch.randn(2, B, hkv, cap, d, generator=g, device=DEV).to(torch.bfloat16)
    inv = 10000.0 ** (-2 * torch.arange(d // 2, dtype=F64, device=DEV) / d)
    words = (mn + 31) // 32

    def inputs(seed):
        r = np.random.RandomState(seed)
        n = [0] * B
        for _ in range(tokens - 5 * seed):  # some of the buffers' tokens belong to nobody
            n[r.choice([b for b in range(B) if n[b] < mn])] += 1
        T = [k + int(r.randint(0, cap - k + 1)) for k in n]
        masks = [random_tree(k, r) if k else np.zeros((0, 0), bool) for k in n]
        mask = torch.zeros(tokens, words, dtype=torch.int32, device=DEV)
        rows = pack_rows([row for m in masks for row in m], words)
        mask[:rows.shape[0]] = rows
        path, plen = np.zeros((B, mn), np.int32), [0] * B
        for b in range(B):
            if n[b]:
                kept = np.flatnonzero(masks[b][int(r.randint(n[b]))])
                plen[b] = len(kept)
                path[b, :plen[b]] = kept
        pos = i32(r.randint(0, 100000, tokens).tolist())
        gg = torch.Generator(device=DEV).manual_seed(100 + seed)
        qkv = torch.randn(tokens, (hq + 2 * hkv) * d, generator=gg, device=DEV).to(torch.bfloat16)
        return [i32(starts(n)), i32(T), pos, mask, i32(path), i32(plen), qkv]

    def buffers():
        kv = first.clone()
        return dict(kv=kv, caches=torch.tensor([kv[0].data_ptr(), kv[1].data_ptr()], dtype=torch.int64, device=DEV),
                    Q=torch.zeros(tokens, hq, d, dtype=torch.bfloat16, device=DEV),
                    out=torch.zeros(tokens, hq, d, dtype=torch.bfloat16, device=DEV),
                    new_len=torch.zeros(B, dtype=torch.int32, device=DEV), ws=tb.workspace(256),
                    wt=tb.workspace(tb.tree_attn_workspace_bytes(dm, tokens, mn)))

    def step(x, y):
        qb, T, pos, mask, path, plen, qkv = x
        K, V = y["kv"][0], y["kv"][1]
        tb.norm_rope_append(dm, qkv, qb, T, pos, None, None, 0.0, inv, True, y["Q"], K, V, y["ws"])
        tb.tree_attn(dm, y["Q"], K, V, qb, mn, T, mask, 1 / math.sqrt(d), y["out"], y["wt"])
        tb.tree_accept(dm, 1, y["caches"], qb, T, path, plen, y["new_len"], y["ws"])

    x, y = inputs(0), buffers()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(x, y)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (3, 0, 7):
        new, want = inputs(seed), buffers()
        step(new, want)
        for a, b in zip(x, new):
            a.copy_(b)
        y["kv"].copy_(first)
        for name in ("Q", "out", "new_len"):
            y[name].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("kv", "Q", "out", "new_len"):
            assert torch.equal(y[name], want[name]), (seed, name)
        for w in (y["ws"], y["wt"], want["ws"], want["wt"]):
            assert tb.workspace_check(w) == 0
        assert bool((want["new_len"] <= new[1]).all()) and not bool((want["out"] == 0).all())


# ------------------------------------------------------------------ a run of them together

def test_prompt_tree_accept_decode_together():
    """A prompt in two chunks, a drafted tree, its accepted path, and the decode
    step behind it, against one 64-bit model of the whole sequence."""
    B, hq, hkv, d, cap, L = 2, 8, 2, 64, 448, 2
    chunks, nodes = [[130, 40], [57, 200]], [9, 30]
    g = torch.Generator(device=DEV).manual_seed(11)
    r = np.random.RandomState(11)
    dm = tb.dims(B, hq, hkv, d, 16, cap)
    inv = 500000.0 ** (-2 * torch.arange(d // 2, dtype=F64, device=DEV) / d)
    qw = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
    kw = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
    kv = torch.full((L, 2, B, hkv, cap, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    step = B * hkv * cap * d * 2
    caches = torch.tensor([kv.data_ptr() + i * step for i in range(2 * L)], dtype=torch.int64, device=DEV)
    wsr, scale = tb.workspace(256), 1 / math.sqrt(d)
    T = [0, 0]

    def feed(n, pos, attend):
        for b in range(B):
            T[b] += n[b]
        total, outs = sum(n), []
        for l in range(L):
            qkv = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device=DEV).to(torch.bfloat16)
            Q = torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEV)
            tb.norm_rope_append(dm, qkv, i32(starts(n)), i32(T), pos, qw, kw, 1e-6, inv, False, Q, kv[l, 0], kv[l, 1], wsr)
            outs.append((Q, attend(Q, kv[l, 0], kv[l, 1])))
        return outs

    for c in range(2):
        n = [chunks[0][c], chunks[1][c]]

        def attend(Q, K, V):
            out = torch.zeros_like(Q)
            ws = tb.workspace(tb.prompt_attn_workspace_bytes(dm, Q.shape[0], max(n)))
            tb.prompt_attn(dm, Q, K, V, i32(starts(n)), max(n), i32(T), scale, out, ws)
            assert tb.workspace_check(ws) == 0
            return out

        for l, (Q, out) in enumerate(feed(n, None, attend)):
            check(out, *reference(Q, kv[l, 0], kv[l, 1], n, T, scale, causal(n, T)), f"chunk {c} layer {l}")

    n, before = nodes, list(T)
    masks = [random_tree(k, r) for k in n]
    depth = np.concatenate([before[b] + masks[b].sum(1) - 1 for b in range(B)])
    mask = pack_rows([row for m in masks for row in m], 1)

    def attend_tree(Q, K, V):
        out = torch.zeros_like(Q)
        ws = tb.workspace(tb.tree_attn_workspace_bytes(dm, Q.shape[0], max(n)))
        tb.tree_attn(dm, Q, K, V, i32(starts(n)), max(n), i32(T), mask, scale, out, ws)
        assert tb.workspace_check(ws) == 0
        return out

    for l, (Q, out) in enumerate(feed(n, i32(depth), attend_tree)):
        check(out, *reference(Q, kv[l, 0], kv[l, 1], n, T, scale, tree_see(masks, n, T)), f"tree layer {l}")

    # accept each tree's deepest path: its rows then read as if they had been decoded one by one
    paths = [np.flatnonzero(m[int(m.sum(1).argmax())]) for m in masks]
    want = [[kv[:, :, b, :, :before[b]].clone(), kv[:, :, b][:, :, :, before[b] + torch.tensor(paths[b], device=DEV)].clone()]
            for b in range(B)]
    path = np.zeros((B, 32), dtype=np.int32)
    for b in range(B):
        path[b, :len(paths[b])] = paths[b]
    new_len = torch.zeros(B, dtype=torch.int32, device=DEV)
    tb.tree_accept(dm, L, caches, i32(starts(n)), i32(T), i32(path), i32([len(p) for p in paths]), new_len, wsr)
    T = [before[b] + len(paths[b]) for b in range(B)]
    assert new_len.tolist() == T
    for b in range(B):
        assert torch.equal(kv[:, :, b, :, :before[b]], want[b][0])
        assert torch.equal(kv[:, :, b, :, before[b]:T[b]], want[b][1])

    # the decode loop goes on behind it
    def attend_decode(Q, K, V):
        out = torch.zeros(B, hq, d, device=DEV)
        ws = tb.workspace(tb.attn_workspace_bytes(dm))
        tb.decode_attn(dm, Q, K, V, i32(T), scale, out, ws)
        assert tb.workspace_check(ws) == 0
        return out

    for l, (Q, out) in enumerate(feed([1, 1], None, attend_decode)):
        check(out, *reference(Q, kv[l, 0], kv[l, 1], [1, 1], T, scale, causal([1, 1], T)), f"decode layer {l}")
    assert tb.workspace_check(wsr) == 0


# ------------------------------------------------------------------ streams

def test_calls_on_a_side_stream_wait_for_it_only():
    n, T = [64, 64], [900, 64]
    Q, K, V, out, scale = run_prompt(n, T, 8, 2, 64, seed=12, extra=0)
    dm = tb.dims(2, 8, 2, 64, 16, K.shape[2])
    ws = tb.workspace(tb.prompt_attn_workspace_bytes(dm, 128, 64))
    got = torch.zeros_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Q2 = torch.zeros_like(Q)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        Q2.copy_(Q)                        # written on the side stream, behind the sleep
        tb.prompt_attn(dm, Q2, K, V, i32(starts(n)), 64, i32(T), scale, got, ws, stream=side)
    side.synchronize()
    assert torch.equal(got, out)


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("n,T", [([40], [40]), ([150, 20], [700, 20]), ([60], [9000])])
def test_non_finite_rows_reach_only_the_tokens_that_see_them(n, T, tree, d):
    """A NaN or an infinity in a new token's K or V row changes the tokens that
    attend to it, and no other."""
    hq, hkv = 8, 2
    g = torch.Generator(device=DEV).manual_seed(21)
    r = np.random.RandomState(21)
    cap = (max(T) + 127) // 128 * 128
    K, V = make_cache(g, len(n), hkv, cap, d, T)
    Q = torch.randn(sum(n), hq, d, generator=g, device=DEV).to(torch.bfloat16)
    Kc, Vc = K.clone(), V.clone()
    at = {}                                   # (sequence, new token) -> what is odd about its row
    for b in range(len(n)):
        for j, kind in ((n[b] // 3, "V nan"), (n[b] // 2, "V inf"), (n[b] - 2, "K nan"), (n[b] - 1, "V nan")):
            row = T[b] - n[b] + j
            at[b, j] = kind
            if kind == "K nan":
                K[b, :, row, 5] = float("nan")
                Kc[b, :, row] = 0
            else:
                V[b, :, row, 7] = float("nan") if kind == "V nan" else float("inf")
                Vc[b, :, row, 7] = 0
    masks = [random_tree(k, r) if tree else np.tril(np.ones((k, k), dtype=bool)) for k in n]
    if tree:
        for m in masks:                       # the first odd row is no ancestor of most
            m[m.shape[0] // 3 + 2:, m.shape[0] // 3] = False
    out = torch.zeros_like(Q)
    dm, scale = tb.dims(len(n), hq, hkv, d, 16, cap), 1 / math.sqrt(d)
    size = tb.tree_attn_workspace_bytes if tree else tb.prompt_attn_workspace_bytes
    ws = tb.workspace(size(dm, sum(n), max(n)))
    if tree:
        mask = pack_rows([row for m in masks for row in m], (max(n) + 31) // 32)
        mask = mask if mask.shape[1] else None
        tb.tree_attn(dm, Q, K, V, i32(starts(n)), max(n), i32(T), mask, scale, out, ws)
    else:
        tb.prompt_attn(dm, Q, K, V, i32(starts(n)), max(n), i32(T), scale, out, ws)
    assert tb.workspace_check(ws) == 0
    ref, tol = reference(Q, Kc, Vc, n, T, scale, tree_see(masks, n, T))
    s = starts(n)
    clean = 0
    for b in range(len(n)):
        for i in range(n[b]):
            seen = {kind for (bb, j), kind in at.items() if bb == b and masks[b][i, j]}
            o, x = out[s[b] + i], slice(s[b] + i, s[b] + i + 1)
            if "K nan" in seen:
                assert o.isnan().all(), (b, i)
                continue
            if "V nan" in seen:
                assert o[:, 7].isnan().all(), (b, i)
            elif "V inf" in seen:
                assert (o[:, 7] == float("inf")).all(), (b, i)
            keep = [c for c in range(d) if c != 7 or not seen]
            check(out[x][..., keep], ref[x][..., keep], tol[x][..., keep], f"token {b, i}")
            clean += not seen
    assert clean >= sum(n) // 4


def test_prompt_logits_far_apart():
    """Logits that rise by hundreds along the context (the running reference
    is raised again and again), and ones that fall by as much."""
    n, T, d = [130, 70], [900, 2000], 128
    g = torch.Generator(device=DEV).manual_seed(31)
    K, V = make_cache(g, 2, 2, 2048, d, T, heavy=False)
    Q = torch.randn(200, 8, d, generator=g, device=DEV).to(torch.bfloat16)
    u = torch.randn(d, generator=g, device=DEV)
    Q = (Q.float() * 0.1 + u).to(torch.bfloat16)
    for sign in (1, -1):
        ramp = sign * torch.linspace(-4, 4, 2048, device=DEV)[None, None, :, None]
        Kr = (K.float() * 0.1 + ramp * u).to(torch.bfloat16)
        for b in range(2):
            Kr[b, :, T[b]:] = float("nan")
        _, _, _, out, scale = run_prompt(n, T, 8, 2, d, extra=0, K=Kr, V=V, Q=Q, cap=2048)
        ref, tol = reference(Q, Kr, V, n, T, scale, causal(n, T))
        check(out, ref, tol, f"sign {sign}")


# ------------------------------------------------------------------ what the binding refuses

def test_binding_refuses_types_shapes_and_layouts():
    d = tb.dims(2, 8, 2, 64, 16, 32)
    z = lambda *s, t=torch.bfloat16, dev=DEV: torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
    good = dict(Q=z(3, 8, 64), K=z(2, 2, 32, 64), V=z(2, 2, 32, 64), q_begin=i32([0, 1, 3]), ctx_len=i32([1, 2]),
                out=z(3, 8, 64), mask=z(3, 1, t=torch.int32), ws=tb.workspace(1 << 22), qkv=z(3, 12 * 64),
                inv=torch.ones(32, dtype=F64, device=DEV), pos=i32([0, 1, 2]), w=z(64), caches=z(2, t=torch.int64),
                path=z(2, 4, t=torch.int32), plen=i32([0, 0]), new=i32([0, 0]))

    def prompt(**kw):
        a = {**good, **kw}
        tb.prompt_attn(d, a["Q"], a["K"], a["V"], a["q_begin"], kw.get("mx", 2), a["ctx_len"], kw.get("scale", 0.1),
                       a["out"], a["ws"])

    def tree(**kw):
        a = {**good, **kw}
        tb.tree_attn(d, a["Q"], a["K"], a["V"], a["q_begin"], 2, a["ctx_len"], a["mask"], 0.1, a["out"], a["ws"])

    def rope(**kw):
        a = {**good, **kw}
        tb.norm_rope_append(d, a["qkv"], a["q_begin"], a["ctx_len"], a["pos"], a["w"], a["w"], 1e-6, a["inv"], False,
                            a["Q"], a["K"], a["V"], a["ws"])

    def accept(**kw):
        a = {**good, **kw}
        tb.tree_accept(d, 1, a["caches"], a["q_begin"], a["ctx_len"], a["path"], a["plen"], a["new"], a["ws"])

    for call, odd in [
        (prompt, dict(Q=z(3, 8, 64, t=torch.float16))), (prompt, dict(Q=z(3, 4, 64))), (prompt, dict(Q=z(3, 512))),
        (prompt, dict(K=z(2, 2, 31, 64))), (prompt, dict(V=z(2, 2, 64, 32).transpose(2, 3))),
        (prompt, dict(q_begin=i32([0, 3]))), (prompt, dict(q_begin=i32([0, 1, 3]).long())),
        (prompt, dict(ctx_len=i32([1, 2]).cpu())), (prompt, dict(out=z(4, 8, 64))), (prompt, dict(out=z(3, 8, 64, t=torch.float32))),
        (prompt, dict(out=good["Q"])), (prompt, dict(mx=0)), (prompt, dict(mx=1 << 40)), (prompt, dict(scale=0.0)),
        (prompt, dict(ws=tb.workspace(1 << 22).cpu())), (prompt, dict(Q="no tensor")),
        (tree, dict(mask=z(3, 2, t=torch.int32))), (tree, dict(mask=z(3, 1, t=torch.int64))), (tree, dict(mask=None)),
        (rope, dict(qkv=z(3, 11 * 64))), (rope, dict(qkv=z(12 * 64, 3).t())), (rope, dict(qkv=z(3, 12 * 64, t=torch.float32))),
        (rope, dict(pos=i32([0, 1]))), (rope, dict(w=z(32))), (rope, dict(inv=torch.ones(32, device=DEV))),
        (rope, dict(inv=torch.ones(36, dtype=F64, device=DEV))), (rope, dict(K=z(2, 2, 32, 32))),
        (accept, dict(caches=z(4, t=torch.int64))), (accept, dict(path=z(4, t=torch.int32))),
        (accept, dict(new=good["ctx_len"])), (accept, dict(plen=i32([0]))),
    ]:
        with pytest.raises(tb.TbError):
            call(**odd)
    prompt(), tree(), rope(), accept()         # and takes what is right
    with pytest.raises(TypeError):
        tb.prompt_attn(d, good["Q"], good["K"], good["V"], good["q_begin"], 2, good["ctx_len"], "0.1", good["out"], good["ws"])
    torch.cuda.synchronize()
    assert tb.workspace_check(good["ws"]) in (0, _lib.TB_FLAG_BAD_CACHE)   # (accept's cache addresses are null)


def test_calls_of_no_tokens_do_nothing():
    d = tb.dims(2, 8, 2, 64, 16, 32)
    K = torch.randn(2, 2, 32, 64, device=DEV).to(torch.bfloat16)
    V, want = K.clone(), K.clone()
    Q = torch.zeros(0, 8, 64, dtype=torch.bfloat16, device=DEV)
    ws = tb.workspace(tb.prompt_attn_workspace_bytes(d, 0, 1))
    qb, ctx = i32([0, 0, 0]), i32([0, 0])
    tb.prompt_attn(d, Q, K, V, qb, 1, ctx, 0.1, torch.zeros_like(Q), ws)
    tb.tree_attn(d, Q, K, V, qb, 1, ctx, torch.zeros(0, 1, dtype=torch.int32, device=DEV), 0.1, torch.zeros_like(Q), ws)
    tb.norm_rope_append(d, torch.zeros(0, 12 * 64, dtype=torch.bfloat16, device=DEV), qb, ctx, None, None, None, 0.0, None,
                        False, Q, K, V, ws)
    torch.cuda.synchronize()
    assert tb.workspace_check(ws) == 0 and torch.equal(K, want) and torch.equal(V, want)


# ------------------------------------------------------------------ many sequences, long caches

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
def test_more_sequences_than_a_warp_looks_at_once(tree, d):
    r = np.random.RandomState(40 + d)
    n = [int(x) for x in r.choice([0, 1, 2, 5, 40, 70], 100)]
    T = [k + int(x) for k, x in zip(n, r.choice([0, 3, 200, 700], 100))]
    if tree:
        masks = [random_tree(k, r) for k in n]
        Q, K, V, out, scale = run_tree(n, T, masks, 8, 2, d, seed=1)
        see = tree_see(masks, n, T)
    else:
        Q, K, V, out, scale = run_prompt(n, T, 8, 2, d, seed=1)
        see = causal(n, T)
    ref, tol = reference(Q, K, V, n, T, scale, see)
    check(out[:sum(n)], ref[:sum(n)], tol[:sum(n)])


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: the last (sequence, KV head) lies
    past 4 GB of each of K and V, for the write, both attentions and the move."""
    hq, hkv, d, cap = 4, 4, 128, (1 << 22)
    assert hkv * cap * d >= 1 << 31
    T, n = cap - 5, 6
    g = torch.Generator(device=DEV).manual_seed(50)
    kv = torch.zeros(1, 2, 1, hkv, cap, d, dtype=torch.bfloat16, device=DEV)
    K, V = kv[0, 0], kv[0, 1]
    lo = T - 3000                              # everything before has the same small key and zero value
    K[..., :lo, :] = 0.125
    K[:, :, lo:T] = torch.randn(1, hkv, 3000, d, generator=g, device=DEV).to(torch.bfloat16)
    V[:, :, lo:T] = torch.randn(1, hkv, 3000, d, generator=g, device=DEV).to(torch.bfloat16)
    dm = tb.dims(1, hq, hkv, d, 16, cap)
    qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g, device=DEV).to(torch.bfloat16)
    Q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device=DEV)
    qb, ctx, ws = i32([0, n]), i32([T]), tb.workspace(256)
    tb.norm_rope_append(dm, qkv, qb, ctx, None, None, None, 0.0, None, False, Q, K, V, ws)
    x = qkv.view(n, 3 * hkv, d)
    assert torch.equal(K[0, :, T - n:T], x[:, hkv:2 * hkv].transpose(0, 1))
    assert torch.equal(V[0, :, T - n:T], x[:, 2 * hkv:].transpose(0, 1)) and torch.equal(Q, x[:, :hkv])
    scale = 0.05
    mask = pack_rows(np.tril(np.ones((n, n), dtype=bool)), 1)
    outs = []
    for tree in (False, True):
        out = torch.zeros_like(Q)
        size = tb.tree_attn_workspace_bytes if tree else tb.prompt_attn_workspace_bytes
        wsa = tb.workspace(size(dm, n, n))
        if tree:
            tb.tree_attn(dm, Q, K, V, qb, n, ctx, mask, scale, out, wsa)
        else:
            tb.prompt_attn(dm, Q, K, V, qb, n, ctx, scale, out, wsa)
        assert tb.workspace_check(wsa) == 0
        outs.append(out)
    assert torch.equal(*outs)
    # the rows before `lo` share one logit: lo times its weight in the denominator
    for i in range(n):
        end = T - n + i + 1
        for h in range(hkv):
            q = Q[i, h].to(F64)
            k, v = K[0, h, lo:end].to(F64), V[0, h, lo:end].to(F64)
            l = torch.cat([(q.sum() * 0.125)[None], k @ q]) * scale
            p = torch.exp(l - l.max())
            p[0] *= lo
            ref, A = (p[1:] @ v) / p.sum(), (p[1:] @ v.abs()) / p.sum()
            # fp32 sums of 2^22 terms, 128 at a time: the adds of a row's tiles, 2^15 e, and what `check` counts
            tol = U * ref.abs() + A * (U + 2 * (2.0 ** -21 + 256 * E * 10) + 2 * E * 2 ** 15)
            check(outs[0][i, h], ref, tol, f"token {i} head {h}")
    before = kv[0, :, 0, :, T - n:T].clone()
    new_len = torch.zeros(1, dtype=torch.int32, device=DEV)
    caches = torch.tensor([K.data_ptr(), V.data_ptr()], dtype=torch.int64, device=DEV)
    tb.tree_accept(dm, 1, caches, qb, ctx, i32([[1, 2, 5]]), i32([3]), new_len, ws)
    assert tb.workspace_check(ws) == 0 and new_len.item() == T - n + 3
    assert torch.equal(kv[0, :, 0, :, T - n:T - n + 3], before[:, :, [1, 2, 5]])
    assert torch.equal(kv[0, :, 0, :, T - n + 3:T], before[:, :, 3:])


def test_two_streams_at_once_with_workspaces_of_their_own():
    cases = [([64, 9], [3000, 40], 128), ([200], [200], 64), ([5, 5, 5], [900, 2000, 5], 128)]
    runs, streams = [], [torch.cuda.Stream() for _ in cases]
    for k, (n, T, d) in enumerate(cases):
        Q, K, V, out, scale = run_prompt(n, T, 8, 2, d, seed=60 + k, extra=0)
        dm = tb.dims(len(n), 8, 2, d, 16, K.shape[2])
        runs.append((dm, Q, K, V, i32(starts(n)), max(n), i32(T), scale, out,
                     tb.workspace(tb.prompt_attn_workspace_bytes(dm, sum(n), max(n))), torch.zeros_like(out)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (dm, Q, K, V, qb, mx, ct, scale, out, ws, got) in zip(streams, runs):
            tb.prompt_attn(dm, Q, K, V, qb, mx, ct, scale, got, ws, stream=s)
    torch.cuda.synchronize()
    for dm, Q, K, V, qb, mx, ct, scale, out, ws, got in runs:
        assert torch.equal(got, out) and tb.workspace_check(ws) == 0
