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

__device__ __forceinline__ void unpack4(uint2 u, float *f) {
    f[0] = bf16_lo(u.x);
    f[1] = bf16_hi(u.x);
    f[2] = bf16_lo(u.y);
    f[3] = bf16_hi(u.y);
}
__device__ __forceinline__ uint2 pack4(const float *f) {
    uint2 u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(f[1]), "f"(f[0]));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(f[3]), "f"(f[2]));
    return u;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
norm_rope_append_kernel(const RopeParams p) {
    constexpr int LPH = D / 8;    // lanes per head row
    constexpr int HPI = 32 / LPH; // head rows per warp instruction
    constexpr int kUnroll = 4;
    const int lane = threadIdx.x & 31;
    const int warps_per_token = (p.Hq + 2 * p.Hkv + p.heads_per_warp - 1) / p.heads_per_warp;
    griddep_wait();
    griddep_launch_dependents();
    const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int tok = (int)(w / warps_per_token);
    if (tok >= p.n_tokens) return;
    const int h0 = (int)(w % warps_per_token) * p.heads_per_warp;
    const int h1 = min(h0 + p.heads_per_warp, p.Hq + 2 * p.Hkv);
    const int b = find_seq(p.q_begin, p.batch, tok, lane);
    if (b < 0) return;
    const SeqSpan sp = seq_span(p.q_begin, b, p.n_tokens);
    if (tok < sp.begin || tok >= sp.begin + sp.n) return;  // behind the last sequence
    const int row = p.ctx_len[b] - sp.n + (tok - sp.begin);
    const bool cached = row >= 0 && row < p.cap;
    if (!cached && h0 == 0 && lane == 0) raise_flag(p.flags, TB_FLAG_CTX_RANGE);

    // this lane's two groups of 4 values: half style pairs group r with group
    // r + R (R = rot / 8); interleaved pairs lie within a group
    const int l = lane % LPH, R = p.rot / 8;
    int ga, gb;
    bool ra, rb;  // does the group turn?
    if (p.interleaved) {
        ga = 2 * l;
        gb = 2 * l + 1;
        ra = ga * 4 < p.rot;
        rb = gb * 4 < p.rot;
    } else {
        ra = rb = l < R;
        ga = l < R ? l : l + R;
        gb = l < R ? l + R : l + LPH;
    }
    // cosines and sines of the lane's 4 pairs: the HPI lanes that hold the same
    // values of different heads work out 4 / HPI of them each and trade
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (h0 < p.Hq + p.Hkv && p.rot > 0) {
        const double P = (double)(p.pos ? p.pos[tok] : row);
        float c[4 / HPI], s[4 / HPI];
#pragma unroll
        for (int i = 0; i < 4 / HPI; ++i) {
            const int j = 4 * l + i * HPI + lane / LPH;  // the pair's frequency
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

    const uint16_t *src = p.qkv + (size_t)tok * p.row_stride;
    const size_t kv0 = ((size_t)b * p.Hkv * p.cap + (cached ? row : 0)) * D;
    for (int hb = h0; hb < h1; hb += HPI * kUnroll) {
        uint2 ua[kUnroll], ub[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = hb + u * HPI + lane / LPH;
            ua[u] = ub[u] = make_uint2(0u, 0u);
            if (h < h1) {
                const uint2 *r = reinterpret_cast<const uint2 *>(src + (size_t)h * D);
                ua[u] = r[ga];
                ub[u] = r[gb];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = hb + u * HPI + lane / LPH;
            const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
            uint2 oa = ua[u], ob = ub[u];
            if (hb + u * HPI < p.Hq + p.Hkv) {  // (uniform: some head of the warp is q or k)
                float a[4], c[4];
                unpack4(oa, a);
                unpack4(ob, c);
                if (p.qw || p.kw) {
                    float ss = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) ss = fmaf(a[k], a[k], fmaf(c[k], c[k], ss));
#pragma unroll
                    for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
                    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                    const uint2 *wr = reinterpret_cast<const uint2 *>(is_q ? p.qw : p.kw);
                    if (wr) {
                        float wa[4], wb[4];
                        unpack4(__ldg(wr + ga), wa);
                        unpack4(__ldg(wr + gb), wb);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            a[k] *= inv * wa[k];
                            c[k] *= inv * wb[k];
                        }
                    }
                }
                if (p.interleaved) {
                    if (ra) {
                        const float x0 = a[0], x1 = a[1], x2 = a[2], x3 = a[3];
                        a[0] = x0 * cs[0] - x1 * sn[0];
                        a[1] = x1 * cs[0] + x0 * sn[0];
                        a[2] = x2 * cs[1] - x3 * sn[1];
                        a[3] = x3 * cs[1] + x2 * sn[1];
                    }
                    if (rb) {
                        const float x0 = c[0], x1 = c[1], x2 = c[2], x3 = c[3];
                        c[0] = x0 * cs[2] - x1 * sn[2];
                        c[1] = x1 * cs[2] + x0 * sn[2];
                        c[2] = x2 * cs[3] - x3 * sn[3];
                        c[3] = x3 * cs[3] + x2 * sn[3];
                    }
                } else if (ra) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x = a[k], y = c[k];
                        a[k] = x * cs[k] - y * sn[k];
                        c[k] = y * cs[k] + x * sn[k];
                    }
                }
                if (is_q || is_k) {
                    oa = pack4(a);
                    ob = pack4(c);
                }
            }
            if (h >= h1 || (!is_q && !cached)) continue;
            uint16_t *dst;
            if (is_q)
                dst = p.Q + ((size_t)tok * p.Hq + h) * D;
            else if (is_k)
                dst = p.K + kv0 + (size_t)(h - p.Hq) * p.cap * D;
            else
                dst = p.V + kv0 + (size_t)(h - p.Hq - p.Hkv) * p.cap * D;
            reinterpret_cast<uint2 *>(dst)[ga] = oa;
            reinterpret_cast<uint2 *>(dst)[gb] = ob;
        }
    }
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
    // unless that leaves SMs idle; then one unrolled round of heads each
    const int heads = d.n_q_heads + 2 * d.n_kv_heads;
    const int round = 4 * (32 / (d.head_dim / 8));
    p.heads_per_warp = n_tokens >= num_sms() * 16 ? heads : round;
    const long long warps = (long long)n_tokens * ((heads + p.heads_per_warp - 1) / p.heads_per_warp);
    const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    if (d.head_dim == 128) return launch_pdl(norm_rope_append_kernel<128>, grid, dim3(kThreads), 0, st, p);
    return launch_pdl(norm_rope_append_kernel<64>, grid, dim3(kThreads), 0, st, p);
}

}  // namespace tb
