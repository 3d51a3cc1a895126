// tb_norm_rope_append: per-head RMS norms of queries and keys and the rotary
// position rotation in one pass over the projected rows, writing the queries
// packed and the keys and values straight into the cache.
//
// For a head row x (d values) of token i of sequence b at position P:
//
//   y = x * w / sqrt(mean(x^2) + eps)                     (norm; without weights y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)   for each rotated pair
//
// with the angle P * inv_freq[j] of pair j.  The product is taken in fp64 and
// reduced to a fraction of a half turn before it is rounded to fp32: at
// position 2^20 an fp32 product alone would be off by up to 2^-4 radians.
// Everything else is fp32 with one rounding to bf16 at the end.
//
// The pass moves (Hq + 2 Hkv) * d values in and out per token and computes a
// few operations on each, so it is bound by memory; small calls are bound by
// their latency.  A head row is held by d/8 lanes, each with two groups of 4
// values that pair up within the lane, so the rotation needs no exchange and
// the norm one reduction over the lanes.  A lane keeps the 4 (cos, sin) pairs
// of its values in registers for all of the token's heads.
//
// On a B200, 32 query and 8 KV heads of 128: 32K tokens (805 MB moved) 126 us
// in a graph, 6.4 TB/s or 0.97 of a plain copy, and 134 to 138 in a loop of
// calls (0.90); 16 tokens 3.1 us, the launch.  24 heads of 64: 13.2 us for 8.4K
// tokens (52 MB), 22.2 for 16.9K, 40.9 for 33.8K, that is 3.5 us and 5.5 TB/s,
// whether of one sequence or eight and with 4 or 16 of the pairs turned.
#include "common.cuh"
#include "internal.h"
#include "multi.h"

namespace tb {
namespace {

constexpr int kThreads = 128;
constexpr uint32_t kFullMask = 0xffffffffu;

struct RopeParams {
    const uint16_t *qkv;
    long long row_stride;
    const int32_t *q_begin, *ctx_len, *pos;
    const uint16_t *qw, *kw;
    const double *inv_freq;
    uint16_t *Q, *K, *V;
    uint32_t *flags;
    float eps;
    int batch, Hq, Hkv, cap, n_tokens, rot, interleaved, heads_per_warp;
};

// The last sequence whose first token is at or before `tok` (of those that
// start at the same token, all but the last are empty); -1 if none.  All
// lanes take part: each round narrows the range 32-fold.
__device__ __forceinline__ int find_seq(const int32_t *q_begin, int batch, int tok, int lane) {
    int lo = 0, hi = batch;  // q_begin[< lo] <= tok < q_begin[>= hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step - 1;
        const uint32_t le = __ballot_sync(kFullMask, at < hi && q_begin[at] <= tok);
        const int k = __popc(le);  // probes at or before tok (q_begin does not decrease)
        const int nlo = lo + k * step;
        if (step == 1) return nlo - 1;
        hi = min(hi, nlo + step - 1);
        lo = nlo;
    }
    return lo - 1;
}

typedef unsigned long long u64;
__device__ __forceinline__ u64 pack2(float lo, float hi) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(u64 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ u64 sub2(u64 a, u64 b) {
    u64 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A lane's 8 values of a head row as 4 pairs (x_j, y_j) of the rotation, held
// as x_0 x_1 | x_2 x_3 and y_0 y_1 | y_2 y_3: half style pairs value k of the
// first group with value k of the second, interleaved pairs neighbours.
struct Pairs {
    u64 x[2], y[2];
};
template <bool INTER>
__device__ __forceinline__ Pairs unpack_pairs(uint2 a, uint2 b) {
    if constexpr (INTER)
        return {{pack2(bf16_lo(a.x), bf16_lo(a.y)), pack2(bf16_lo(b.x), bf16_lo(b.y))},
                {pack2(bf16_hi(a.x), bf16_hi(a.y)), pack2(bf16_hi(b.x), bf16_hi(b.y))}};
    else
        return {{pack2(bf16_lo(a.x), bf16_hi(a.x)), pack2(bf16_lo(a.y), bf16_hi(a.y))},
                {pack2(bf16_lo(b.x), bf16_hi(b.x)), pack2(bf16_lo(b.y), bf16_hi(b.y))}};
}
template <bool INTER>
__device__ __forceinline__ void pack_pairs(const Pairs &p, uint2 &a, uint2 &b) {
    float x[4], y[4];
    unpack2(p.x[0], x[0], x[1]);
    unpack2(p.x[1], x[2], x[3]);
    unpack2(p.y[0], y[0], y[1]);
    unpack2(p.y[1], y[2], y[3]);
    if constexpr (INTER) {
        a = make_uint2(pack_bf16(x[0], y[0]), pack_bf16(x[1], y[1]));
        b = make_uint2(pack_bf16(x[2], y[2]), pack_bf16(x[3], y[3]));
    } else {
        a = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        b = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
    }
}

template <bool B>
struct Flag {
    static constexpr bool value = B;
};

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads)
norm_rope_append_kernel(const RopeParams p) {
    constexpr int LPH = D / 8;    // lanes per head row
    constexpr int HPI = 32 / LPH; // head rows per warp instruction
    constexpr int kUnroll = 4;
    const int lane = threadIdx.x & 31;
    const int heads = p.Hq + 2 * p.Hkv;
    const int warps_per_token = (heads + p.heads_per_warp - 1) / p.heads_per_warp;
    griddep_wait();
    griddep_launch_dependents();
    const int w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // (the host keeps it below 2^31)
    const int tok = w / warps_per_token;
    if (tok >= p.n_tokens) return;
    const int h0 = (w - tok * warps_per_token) * p.heads_per_warp;
    const int h1 = min(h0 + p.heads_per_warp, heads);

    // this lane's two groups of 4 values: half style pairs group r with group
    // r + R (R = rot / 8) and leaves the groups from 2 R on alone
    const int l = lane % LPH, hl = lane / LPH, R = p.rot / 8;
    const int ga = INTER ? 2 * l : l < R ? l : l + R;
    const int gb = INTER ? 2 * l + 1 : l < R ? l + R : l + LPH;
    const uint2 *src = reinterpret_cast<const uint2 *>(p.qkv + (size_t)tok * p.row_stride);
    uint2 ua[kUnroll], ub[kUnroll];
    auto fetch = [&](int h, int he) {  // rows h, h + HPI, .. below he
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            ua[u] = ub[u] = make_uint2(0u, 0u);
            if (h + u * HPI < he) {
                const uint2 *r = src + (uint32_t)((h + u * HPI) * (D / 4));
                ua[u] = r[ga];
                ub[u] = r[gb];
            }
        }
    };
    // the first rows are on their way while the sequence is looked up
    fetch(h0 + hl, min(h1, h0 < p.Hq ? p.Hq : h0 < p.Hq + p.Hkv ? p.Hq + p.Hkv : heads));

    const int b = find_seq(p.q_begin, p.batch, tok, lane);
    if (b < 0) return;
    const SeqSpan sp = seq_span(p.q_begin, b, p.n_tokens);
    if (tok < sp.begin || tok >= sp.begin + sp.n) return;  // behind the last sequence
    const int row = p.ctx_len[b] - sp.n + (tok - sp.begin);
    const bool cached = row >= 0 && row < p.cap;
    if (!cached && h0 == 0 && lane == 0) raise_flag(p.flags, TB_FLAG_CTX_RANGE);

    // which of the lane's pairs turn (rot is a multiple of 8, so in half style
    // all or none, in interleaved style those of a group alike)
    const bool ra = INTER ? ga * 4 < p.rot : l < R, rb = INTER ? gb * 4 < p.rot : l < R;
    // cosines and sines of the lane's 4 pairs: the HPI lanes that hold the same
    // values of different heads work out 4 / HPI of them each and trade
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (h0 < p.Hq + p.Hkv && p.rot > 0) {
        const double P = (double)(p.pos ? p.pos[tok] : row);
        float c[4 / HPI], s[4 / HPI];
#pragma unroll
        for (int i = 0; i < 4 / HPI; ++i) {
            const int j = 4 * l + i * HPI + hl;  // the pair's frequency
            double t = 0.0;
            if (j < p.rot / 2) t = P * p.inv_freq[j] * 0.31830988618379067154;  // half turns
            t -= 2.0 * rint(0.5 * t);
            sincospif((float)t, &s[i], &c[i]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            cs[k] = __shfl_sync(kFullMask, c[k / HPI], l + LPH * (k % HPI));
            sn[k] = __shfl_sync(kFullMask, s[k / HPI], l + LPH * (k % HPI));
        }
    }

    const u64 c2[2] = {pack2(cs[0], cs[1]), pack2(cs[2], cs[3])}, s2[2] = {pack2(sn[0], sn[1]), pack2(sn[2], sn[3])};

    // the heads in three runs: queries, keys, values; in each kUnroll rows a
    // lane are requested before the first is worked on
    auto run = [&](int begin, int end, uint16_t *out, uint32_t step, auto turn_c, const uint16_t *weight) {
        constexpr bool kTurn = decltype(turn_c)::value;
        const int hb = max(begin, h0), he = min(end, h1);
        if (hb >= he) return;
        Pairs wt{};
        if (kTurn && weight) {
            const uint2 *r = reinterpret_cast<const uint2 *>(weight);
            wt = unpack_pairs<INTER>(__ldg(r + ga), __ldg(r + gb));
        }
        uint2 *dst = reinterpret_cast<uint2 *>(out);
        for (int h = hb + hl; h - hl < he; h += HPI * kUnroll) {
            if (h != h0 + hl) fetch(h, he);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (h - hl + u * HPI >= he) break;  // (the same for all lanes)
                if constexpr (kTurn) {
                    Pairs v = unpack_pairs<INTER>(ua[u], ub[u]);
                    if (weight) {
                        u64 q2 = mul2(v.x[0], v.x[0]);
                        q2 = fma2(v.y[0], v.y[0], q2);
                        q2 = fma2(v.x[1], v.x[1], q2);
                        q2 = fma2(v.y[1], v.y[1], q2);
                        float s0, s1;
                        unpack2(q2, s0, s1);
                        float ss = s0 + s1;
#pragma unroll
                        for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
                        const float inv = rsqrtf(fmaf(ss, 1.f / D, p.eps));
                        const u64 inv2 = pack2(inv, inv);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            v.x[i] = mul2(mul2(v.x[i], inv2), wt.x[i]);
                            v.y[i] = mul2(mul2(v.y[i], inv2), wt.y[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // (pairs that do not turn keep apart: a NaN in one is no business of the other's)
                        if (INTER ? (i ? rb : ra) : ra) {
                            const u64 x = v.x[i], y = v.y[i];
                            v.x[i] = sub2(mul2(x, c2[i]), mul2(y, s2[i]));
                            v.y[i] = fma2(x, s2[i], mul2(y, c2[i]));
                        }
                    }
                    pack_pairs<INTER>(v, ua[u], ub[u]);
                }
                if (h + u * HPI < he) {
                    uint2 *r = dst + (size_t)(uint32_t)(h + u * HPI - begin) * step;
                    r[ga] = ua[u];
                    r[gb] = ub[u];
                }
            }
        }
    };
    run(0, p.Hq, p.Q + (size_t)tok * p.Hq * D, D / 4, Flag<true>{}, p.qw);
    if (!cached) return;
    const size_t kv0 = ((size_t)b * p.Hkv * p.cap + row) * D;
    const uint32_t kv_step = (uint32_t)p.cap * (D / 4);  // one KV head, in groups (cap <= 2^22)
    run(p.Hq, p.Hq + p.Hkv, p.K + kv0, kv_step, Flag<true>{}, p.kw);
    run(p.Hq + p.Hkv, heads, p.V + kv0, kv_step, Flag<false>{}, nullptr);
}

}  // namespace

cudaError_t launch_norm_rope_append(const tb_dims &d, const uint16_t *qkv, int64_t row_stride, const int32_t *q_begin,
                                    int32_t n_tokens, const int32_t *ctx_len, const int32_t *pos, const uint16_t *qw,
                                    const uint16_t *kw, float eps, const double *inv_freq, int32_t rot_dim,
                                    int32_t style, uint16_t *Q, uint16_t *K, uint16_t *V, void *ws, cudaStream_t st) {
    RopeParams p{};
    p.qkv = qkv;
    p.row_stride = row_stride;
    p.q_begin = q_begin;
    p.ctx_len = ctx_len;
    p.pos = pos;
    p.qw = qw;
    p.kw = kw;
    p.inv_freq = inv_freq;
    p.Q = Q;
    p.K = K;
    p.V = V;
    p.flags = static_cast<uint32_t *>(ws);
    p.eps = eps;
    p.batch = d.batch;
    p.Hq = d.n_q_heads;
    p.Hkv = d.n_kv_heads;
    p.cap = d.ctx_cap;
    p.n_tokens = n_tokens;
    p.rot = rot_dim;
    p.interleaved = style == TB_ROPE_INTERLEAVED;
    // a warp takes all of a token's heads (its angles are worked out once)
    // unless that leaves SMs idle; then one unrolled round of heads each.  With
    // 48 heads of 128: 64 tokens 7.2 us whole, 3.1 in rounds; 2,368: 16.7, 15.4;
    // 2,800: 17.4, 17.5; 3,500: 18.7, 20.8; 8,000: 35.4, 41.8.  The two meet
    // between 2,700 and 3,000 tokens for 24 to 80 heads of 64 or 128.
    const int heads = d.n_q_heads + 2 * d.n_kv_heads;
    const int round = 4 * (32 / (d.head_dim / 8));
    p.heads_per_warp = n_tokens >= num_sms() * 19 ? heads : round;
    const long long warps = (long long)n_tokens * ((heads + p.heads_per_warp - 1) / p.heads_per_warp);
    const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    auto *kernel = d.head_dim == 128 ? (p.interleaved ? norm_rope_append_kernel<128, true> : norm_rope_append_kernel<128, false>)
                                     : (p.interleaved ? norm_rope_append_kernel<64, true> : norm_rope_append_kernel<64, false>);
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, p);
}

}  // namespace tb
