"""Workloads of the operators that take several new tokens of a sequence at once.

Four operators around one KV cache ([batch][Hkv][ctx_cap][d] bf16), each with a
plain form in elementary torch operations and the framework's own call:

  rope    per-head RMS norms of queries and keys, rotary positions, and the
          write of Q (packed) and of the K and V rows (into the cache)
  prompt  causal attention of packed prompts or chunks over the cache
  tree    attention of drafted token trees over the cache
  accept  the accepted path of a drafted tree moved to the front of the draft
          rows, in every layer's cache

Sequence b has n_b new tokens (tokens q_begin[b] .. q_begin[b+1] of the packed
arrays); its length T_b counts them, and token i of b sits at cache row
T_b - n_b + i.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
THETA = 500000.0
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch of 16 (every layer runs it): latency
        dict(name="rope_step_b16", op="rope", batch=16, hq=32, hkv=8, d=128, new_lo=1, new_hi=1, pre_lo=2000,
             pre_hi=8000, cap=8192, norm=True, rot=128, inter=False),
        # ragged chunks of a smaller model, half of each head rotated, interleaved pairs, no norm
        dict(name="rope_ragged_d64", op="rope", batch=8, hq=16, hkv=4, d=64, new_lo=1, new_hi=1800, pre_lo=0,
             pre_hi=2000, cap=4096, norm=False, rot=32, inter=True),
        # a long prompt's tokens of one layer
        dict(name="rope_prompt_32k", op="rope", batch=1, hq=32, hkv=8, d=128, new_lo=32768, new_hi=32768, pre_lo=0,
             pre_hi=0, cap=32896, norm=True, rot=128, inter=False),
        # a handful of short prompts arriving together
        dict(name="prompt_short_ragged", op="prompt", batch=16, hq=8, hkv=2, d=64, new_lo=1, new_hi=300, pre_lo=0,
             pre_hi=0, cap=512),
        # the last chunk of a prompt whose first 64K tokens are in the cache already
        dict(name="prompt_chunk_64k", op="prompt", batch=1, hq=32, hkv=8, d=128, new_lo=100, new_hi=100,
             pre_lo=65536, pre_hi=65536, cap=65792),
        # an ordinary prompt of 8K tokens
        dict(name="prompt_8k", op="prompt", batch=1, hq=32, hkv=8, d=128, new_lo=8192, new_hi=8192, pre_lo=0,
             pre_hi=0, cap=8320),
        # ragged prompts with cached prefixes, packed
        dict(name="prompt_ragged_d64", op="prompt", batch=5, hq=16, hkv=4, d=64, new_lo=500, new_hi=5000, pre_lo=0,
             pre_hi=3001, cap=8192),
        # the longest prompt
        dict(name="prompt_32k", op="prompt", batch=1, hq=32, hkv=8, d=128, new_lo=32768, new_hi=32768, pre_lo=0,
             pre_hi=0, cap=32896),
        # a drafted tree of one sequence at the 64K context the decode benchmark runs
        dict(name="tree_64k", op="tree", batch=1, hq=32, hkv=8, d=128, new_lo=26, new_hi=26, pre_lo=65536,
             pre_hi=65536, cap=65792),
        # drafted trees of a ragged batch of 16 (the batched benchmark's contexts)
        dict(name="tree_batch16", op="tree", batch=16, hq=32, hkv=8, d=128, new_lo=10, new_hi=60, pre_lo=16384,
             pre_hi=32000, cap=32896),
        # after the verification: one sequence, 32 layers
        dict(name="accept_b1", op="accept", layers=32, batch=1, hkv=8, d=128, new_lo=26, new_hi=26, pre_lo=2000,
             pre_hi=2000, cap=2048),
        # the same for a batch of 16
        dict(name="accept_b16", op="accept", layers=32, batch=16, hkv=8, d=128, new_lo=10, new_hi=60, pre_lo=0,
             pre_hi=190, cap=256),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "tree", "tree", "accept"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * 4
    if op == "accept":
        batch = _logint(rng, 1, 16)
        hi = _logint(rng, 2, 64)
        pre = _logint(rng, 1, 1500)
        cap = -(-(pre + hi) // 32) * 32
        layers = _logint(rng, 1, max(1, min(32, (1 << 21) // (batch * hkv * cap))))
        return dict(op=op, layers=layers, batch=batch, hkv=hkv, d=d, new_lo=rng.randint(1, hi), new_hi=hi,
                    pre_lo=rng.randint(0, pre), pre_hi=pre, cap=cap)
    if op == "rope":
        total = _logint(rng, 1, 32768)
        batch = _logint(rng, 1, min(16, total))
        hi = max(1, total // batch)
        pre = _logint(rng, 1, 8000)
        rot = d if rng.random() < 0.6 else rng.choice([8, 16, 24, 32, 48, 56])
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, new_lo=rng.randint(1, hi), new_hi=hi,
                    pre_lo=rng.randint(0, pre), pre_hi=pre, cap=-(-(pre + hi) // 128) * 128,
                    norm=rng.random() < 0.7, rot=rot, inter=rng.random() < 0.3)
    if op == "tree":
        batch = _logint(rng, 1, 16)
        hi = _logint(rng, 1, 64)
        pre = _logint(rng, 16, 500000 // batch if batch > 4 else 100000)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, new_lo=rng.randint(1, hi), new_hi=hi,
                    pre_lo=rng.randint(0, pre), pre_hi=pre, cap=-(-(pre + hi) // 64) * 64)
    total = _logint(rng, 1, 24000)
    batch = _logint(rng, 1, min(16, total))
    hi = max(1, total // batch)
    pre = rng.choice([0, 0, _logint(rng, 1, max(1, min(60000, 200000000 // total)))])
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, new_lo=rng.randint(1, hi), new_hi=hi,
                pre_lo=rng.randint(0, pre), pre_hi=pre, cap=-(-(pre + hi) // 128) * 128)


def _lengths(case):
    """New tokens and cached prefix of each sequence (of the case alone: the
    work is the same for every seed)."""
    r = np.random.RandomState(7)
    n = r.randint(case["new_lo"], case["new_hi"] + 1, case["batch"])
    n[0] = case["new_hi"]
    p = r.randint(case["pre_lo"], case["pre_hi"] + 1, case["batch"])
    p[-1] = case["pre_hi"]
    return [int(x) for x in n], [int(x) for x in p]


# ------------------------------------------------------------------ inputs

def _tree(n, r):
    """Parents of a drafted tree in breadth-first order: narrow and deep as
    drafting gives them (a node's parent is among the few before it)."""
    return [-1 if i == 0 else int(r.randint(max(0, i - 1 - i // 2), i)) for i in range(n)]


def _ancestors(parents):
    """Row i: bit j set iff drafted token j is i or an ancestor of i."""
    rows = []
    for i, p in enumerate(parents):
        rows.append((1 << i) | (rows[p] if p >= 0 else 0))
    return rows


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    r = np.random.RandomState(int(seed) % (1 << 31))
    op, B, hkv, d, cap = case["op"], case["batch"], case["hkv"], case["d"], case["cap"]
    n, pre = _lengths(case)
    total = sum(n)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = dict(op=op, case=dict(case), n=n, T=[a + b for a, b in zip(n, pre)], max_new=max(n),
             q_begin=torch.tensor(np.concatenate([[0], np.cumsum(n)]), **i32),
             ctx_len=torch.tensor([a + b for a, b in zip(n, pre)], **i32))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)

    if op == "accept":
        L = case["layers"]
        s["kv"] = normal(L, 2, B, hkv, cap, d)
        step = B * hkv * cap * d * 2
        s["caches"] = torch.tensor([s["kv"].data_ptr() + i * step for i in range(2 * L)], dtype=torch.int64,
                                   device=DEV)
        # the accepted path: from the root down, a random child each time
        path = np.zeros((B, max(n)), dtype=np.int32)
        plen = np.zeros(B, dtype=np.int32)
        for b in range(B):
            par, at, k = _tree(n[b], r), -1, 0
            while True:
                kids = [j for j, p in enumerate(par) if p == at]
                if not kids or (k and r.rand() < 0.15):
                    break
                at = kids[r.randint(len(kids))]
                path[b, k] = at
                k += 1
            plen[b] = k
        s["path"], s["path_len"] = torch.tensor(path, **i32), torch.tensor(plen, **i32)
        s["new_len"] = torch.zeros(B, **i32)
        return s

    hq = case["hq"]
    if op == "rope":
        s["qkv"] = normal(total, (hq + 2 * hkv) * d)
        s["K"], s["V"] = normal(B, hkv, cap, d), normal(B, hkv, cap, d)
        s["Q"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEV)
        s["qw"] = (1 + 0.2 * normal(d)).to(torch.bfloat16) if case["norm"] else None
        s["kw"] = (1 + 0.2 * normal(d)).to(torch.bfloat16) if case["norm"] else None
        s["inv_freq"] = THETA ** (-2.0 * torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEV) / case["rot"])
        return s

    s["Q"] = normal(total, hq, d)
    s["K"], s["V"] = normal(B, hkv, cap, d), normal(B, hkv, cap, d)
    # a hundredth of the keys are heavy hitters, as in the decode workloads
    heavy = torch.rand(B, hkv, cap, 1, generator=g, device=DEV) < 0.01
    s["K"] = torch.where(heavy, s["K"] * 4, s["K"])
    s["out"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device=DEV)
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "tree":
        words = (max(n) + 31) // 32
        rows = [m for b in range(B) for m in _ancestors(_tree(n[b], r))]
        bits = np.array([[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in rows], dtype=np.uint32)
        s["mask"] = torch.tensor(bits.view(np.int32), **i32)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_rope(s):
    c = s["case"]
    hq, hkv, d, rot = c["hq"], c["hkv"], c["d"], c["rot"]
    total = s["qkv"].shape[0]
    tok = torch.arange(total, device=DEV)
    seq = torch.searchsorted(s["q_begin"][1:].long(), tok, right=True)
    row = s["ctx_len"].long()[seq] - s["q_begin"].long()[seq + 1] + tok
    ang = row.double()[:, None] * s["inv_freq"]  # 64 bits: far positions turn many times
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    x = s["qkv"].view(total, hq + 2 * hkv, d)

    def turn(h, w):
        y = h.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        if c["inter"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([z, y[..., rot:]], -1).to(torch.bfloat16)

    s["Q"].copy_(turn(x[:, :hq], s["qw"]))
    s["K"][seq, :, row] = turn(x[:, hq:hq + hkv], s["kw"])
    s["V"][seq, :, row] = x[:, hq + hkv:]
    return s["Q"], s["K"], s["V"]


def _plain_attention(s):
    """Both attentions: sequence by sequence, in blocks of queries so that the
    scores of a long prompt fit."""
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G = hq // hkv
    at = 0
    for b, (n, T) in enumerate(zip(s["n"], s["T"])):
        pre = T - n
        for i0 in range(0, n, 2048):
            m = min(2048, n - i0)
            hi = T if c["op"] == "tree" else pre + i0 + m  # no query of the block sees a row at or past hi
            K, V = s["K"][b, :, :hi].float(), s["V"][b, :, :hi].float()
            q = s["Q"][at + i0:at + i0 + m].float().view(m, hkv, G, d).permute(1, 2, 0, 3).reshape(hkv, G * m, d)
            sc = torch.matmul(q, K.transpose(1, 2)).mul_(s["scale"]).view(hkv, G, m, hi)
            col = torch.arange(hi, device=DEV)
            if c["op"] == "tree":
                j = (col - pre).clamp_(min=0)
                word = s["mask"][at + i0:at + i0 + m].long()[:, j // 32]
                see = (((word >> (j % 32)) & 1) == 1) | (col < pre)
            else:
                see = col[None, :] <= pre + i0 + torch.arange(m, device=DEV)[:, None]
            sc.masked_fill_(~see, -math.inf)
            sc.sub_(sc.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(sc.view(hkv, G * m, hi), V).view(hkv, G, m, d) / sc.sum(-1, keepdim=True)
            s["out"][at + i0:at + i0 + m] = o.permute(2, 0, 1, 3).reshape(m, hq, d).to(torch.bfloat16)
        at += n
    return s["out"]


def _plain_accept(s):
    kv, path = s["kv"], s["path"].long()
    base = s["ctx_len"].long() - (s["q_begin"][1:] - s["q_begin"][:-1]).long()
    j = torch.arange(path.shape[1], device=DEV)
    live = j[None] < s["path_len"][:, None]
    dst = (base[:, None] + j)[live]
    src = (base[:, None] + path)[live]
    b = torch.arange(path.shape[0], device=DEV)[:, None].expand_as(live)[live]
    kv[:, :, b, :, dst] = kv[:, :, b, :, src]
    s["new_len"].copy_(base + s["path_len"])
    return kv, s["new_len"]


# ------------------------------------------------------------------ the framework's calls

def _handle(s, tb):
    """Shapes and workspace, which a program keeps beside its buffers."""
    c = s["case"]
    d = tb.dims(c["batch"], c.get("hq", 4 * c["hkv"]), c["hkv"], c["d"], 16, c["cap"])
    if s["op"] == "prompt":
        nbytes = tb.prompt_attn_workspace_bytes(d, s["Q"].shape[0], s["max_new"])
    elif s["op"] == "tree":
        nbytes = tb.tree_attn_workspace_bytes(d, s["Q"].shape[0], s["max_new"])
    else:
        nbytes = 256
    s["dims"], s["ws"] = d, tb.workspace(nbytes)


def _own(s):
    import query_aware_sparse_tb_b200 as tb

    if "ws" not in s:
        _handle(s, tb)
    c, d, ws = s["case"], s["dims"], s["ws"]
    if s["op"] == "rope":
        tb.norm_rope_append(d, s["qkv"], s["q_begin"], s["ctx_len"], None, s["qw"], s["kw"], EPS, s["inv_freq"],
                            c["inter"], s["Q"], s["K"], s["V"], ws)
        return s["Q"], s["K"], s["V"]
    if s["op"] == "prompt":
        tb.prompt_attn(d, s["Q"], s["K"], s["V"], s["q_begin"], s["max_new"], s["ctx_len"], s["scale"], s["out"], ws)
        return s["out"]
    if s["op"] == "tree":
        tb.tree_attn(d, s["Q"], s["K"], s["V"], s["q_begin"], s["max_new"], s["ctx_len"], s["mask"], s["scale"],
                     s["out"], ws)
        return s["out"]
    tb.tree_accept(d, c["layers"], s["caches"], s["q_begin"], s["ctx_len"], s["path"], s["path_len"], s["new_len"], ws)
    return s["kv"], s["new_len"]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "rope":
        return _plain_rope(state)
    if state["op"] == "accept":
        return _plain_accept(state)
    return _plain_attention(state)


# ------------------------------------------------------------------ work

def work(case):
    n, pre = _lengths(case)
    T = [a + b for a, b in zip(n, pre)]
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "accept":
        # the accepted path is random: on average about a sixth of the drafted
        # rows are accepted, each read once and written once
        rows = case["layers"] * 2 * hkv * sum(max(1, x // 6) for x in n)
        return {"bytes": 2.0 * rows * d * 2, "flops": 0.0}
    hq = case["hq"]
    if case["op"] == "rope":
        return {"bytes": 2.0 * sum(n) * (hq + 2 * hkv) * d * 2, "flops": 10.0 * sum(n) * (hq + hkv) * d}
    io = 2.0 * sum(n) * hq * d * 2 + 2.0 * sum(T) * hkv * d * 2
    if case["op"] == "tree":
        return {"bytes": io, "flops": 4.0 * d * hq * sum(a * b for a, b in zip(n, T))}
    return {"bytes": io, "flops": 4.0 * d * hq * sum(a * p + a * (a + 1) / 2 for a, p in zip(n, pre))}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "accept":
        return None  # copies and whole numbers only
    n, T = s["n"], s["T"]
    hkv, d = case["hkv"], case["d"]
    hq = case["hq"]
    G = hq // hkv
    starts = [sum(n[:b]) for b in range(len(n))]
    if case["op"] == "rope":
        rot = case["rot"]
        j = torch.arange(d, device=DEV)
        if case["inter"]:
            partner, freq, sign = j ^ 1, j // 2, torch.where(j % 2 == 0, -1.0, 1.0)
        else:
            partner, freq, sign = (j + rot // 2) % rot, j % (rot // 2), torch.where(j < rot // 2, -1.0, 1.0)
        turned = j < rot
        partner, freq = torch.where(turned, partner, j), torch.where(turned, freq, torch.zeros_like(j))
        Q, K = torch.zeros(s["Q"].shape, dtype=f64, device=DEV), s["K"].to(f64)
        for b in range(len(n)):
            pos = torch.arange(T[b] - n[b], T[b], device=DEV, dtype=f64)
            ang = torch.where(turned, pos[:, None] * s["inv_freq"][freq], torch.zeros((), dtype=f64, device=DEV))
            x = s["qkv"][starts[b]:starts[b] + n[b]].to(f64).view(n[b], hq + 2 * hkv, d)
            for lo, hi, w in ((0, hq, s["qw"]), (hq, hq + hkv, s["kw"])):
                y = x[:, lo:hi]
                if w is not None:
                    y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + EPS) * w.to(f64)
                z = y * ang.cos()[:, None] + sign.to(f64) * y[..., partner] * ang.sin()[:, None]
                if lo == 0:
                    Q[starts[b]:starts[b] + n[b]] = z
                else:
                    K[b, :, T[b] - n[b]:T[b]] = z.transpose(0, 1)
        return Q, K, None
    out = torch.zeros(s["out"].shape, dtype=f64, device=DEV)
    for b in range(len(n)):
        pre = T[b] - n[b]
        drafted = None
        if case["op"] == "tree":
            m = s["mask"][starts[b]:starts[b] + n[b]].cpu().numpy().view(np.uint32)
            drafted = torch.tensor([[(int(m[i, k // 32]) >> (k % 32)) & 1 for k in range(n[b])] for i in range(n[b])],
                                   dtype=torch.bool, device=DEV)
        for h in range(hq):
            k, v = s["K"][b, h // G, :T[b]].to(f64), s["V"][b, h // G, :T[b]].to(f64)
            for i0 in range(0, n[b], 4096):
                i1 = min(n[b], i0 + 4096)
                a = (s["Q"][starts[b] + i0:starts[b] + i1, h].to(f64) * s["scale"]) @ k[:pre + i1 if drafted is None else T[b]].T
                if drafted is None:
                    a[:, pre:] += torch.full((i1, i1), -math.inf, dtype=f64, device=DEV).triu(1)[i0:i1]
                else:
                    a[:, pre:][~drafted[i0:i1]] = -math.inf
                p = torch.exp(a - torch.logsumexp(a, 1, keepdim=True))
                out[starts[b] + i0:starts[b] + i1, h] = p @ v[:a.shape[1]]
    return out
