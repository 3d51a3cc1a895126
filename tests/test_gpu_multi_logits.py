"""Logits far beyond ordinary ones through the prompt and the tree attention.

Queries and keys have one coordinate that is not zero, so the dot products are
exact in fp32, and keys take 32 values at least 2^-7 apart relatively.  Logits
of different keys then differ by more than 2^-8 |l|, against roundings of 2^-23
|l|: from |l| = 2^17 on the softmax is the mean over the rows that share the
largest logit, and every other weight is below 2^-500.  The tied rows have one
weight w.  Counted: w's rounding to bf16 (u), its exponential (2^-21) on both
sides, the fp32 sums of N terms, and the result's rounding (u)."""
import math

import pytest
import torch

import query_aware_sparse_tb_b200 as tb
import test_gpu_multi as multi

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("shares", [False, True])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [17, 24, 28, 29, 30, 31, 32, 33, 40, 60, 100, 120])
def test_large_logits(power, d, tree, shares):
    n, T, hq, hkv = [70, 20], [900, 20], 8, 2
    cap = 16384 if shares else 1024
    g = torch.Generator(device=DEV).manual_seed(power + d)
    K, V = multi.make_cache(g, 2, hkv, cap, d, T, heavy=False)
    K[..., 1:] = 0
    K[..., 0] = (1 + torch.randint(0, 32, K.shape[:3], generator=g, device=DEV) / 32.0) * 2.0 ** (power // 2)
    Q = torch.zeros(90, hq, d, dtype=torch.bfloat16, device=DEV)
    scale = 1 / math.sqrt(d) * 1.37
    sign = torch.randint(0, 2, (90, hq), generator=g, device=DEV) * 2 - 1
    x = (1 + torch.randint(0, 128, (90, hq), generator=g, device=DEV) / 128.0) * 2.0 ** (power - power // 2 + 3)
    Q[..., 0] = sign * x
    for b in range(2):
        K[b, :, T[b]:] = float("nan")
    out = torch.zeros_like(Q)
    dm = tb.dims(2, hq, hkv, d, 16, cap)
    size = (tb.tree_attn_workspace_bytes if tree else tb.prompt_attn_workspace_bytes)(dm, 90, 70)
    assert (size > 256) == shares
    ws, qb, ctx = tb.workspace(size), multi.i32([0, 70, 90]), multi.i32(T)
    if tree:
        causal = multi.pack_rows([[j <= i for j in range(k)] for k in n for i in range(k)], 3)
        tb.tree_attn(dm, Q, K, V, qb, 70, ctx, causal, scale, out, ws)
    else:
        tb.prompt_attn(dm, Q, K, V, qb, 70, ctx, scale, out, ws)
    assert tb.workspace_check(ws) == 0
    at = 0
    for b in range(2):
        see = multi.causal(n, T)(b, 0, n[b])
        for h in range(hq):
            k, v = K[b, h // 4, :T[b], 0].double(), V[b, h // 4, :T[b]].double()
            l = (Q[at:at + n[b], h, 0].double()[:, None] * k).masked_fill(~see, -math.inf)
            p = (l == l.amax(1, keepdim=True)).double()
            N = p.sum(1, keepdim=True)
            ref, A = p @ v / N, p @ v.abs() / N
            tol = multi.U * ref.abs() + A * (multi.U + 2 * 2.0 ** -21 + 2 * multi.E * N)
            multi.check(out[at:at + n[b], h], ref, tol, f"logits of 2^{power}, sequence {b}, head {h}")
        at += n[b]


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_large_and_of_ordinary_logits_in_one_warp(d):
    """The odd heads' logits are near 2^33, the even ones' ordinary: those keep
    the ordinary tolerance."""
    n, T, hq, hkv = [40], [700], 8, 2
    g = torch.Generator(device=DEV).manual_seed(d)
    K, V = multi.make_cache(g, 1, hkv, 768, d, T, heavy=False)
    Q = torch.randn(40, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    K[..., 0] = 1 + torch.randint(0, 32, K.shape[:3], generator=g, device=DEV) / 32.0
    K[0, :, 700:] = float("nan")
    Q[:, 1::2] = 0
    Q[:, 1::2, 0] = 2.0 ** 36
    _, _, _, out, scale = multi.run_prompt(n, T, hq, hkv, d, cap=768, extra=0, K=K, V=V, Q=Q)
    ref, tol = multi.reference(Q, K, V, n, T, scale, multi.causal(n, T))
    multi.check(out[:, ::2], ref[:, ::2], tol[:, ::2], "ordinary rows")
    k, see = K[0, :, :700, 0].double(), multi.causal(n, T)(0, 0, 40)
    for h in range(1, hq, 2):
        l = k[h // 4].expand(40, 700).masked_fill(~see, -math.inf)
        p = (l == l.amax(1, keepdim=True)).double()
        N, v = p.sum(1, keepdim=True), V[0, h // 4, :700].double()
        ref, A = p @ v / N, p @ v.abs() / N
        tol = multi.U * ref.abs() + A * (multi.U + 2 * 2.0 ** -21 + 2 * multi.E * N)
        multi.check(out[:, h], ref, tol, f"large rows, head {h}")
