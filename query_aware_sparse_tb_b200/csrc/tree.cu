// tb_tree_accept: after a drafted tree has been verified, the rows of the
// accepted path move to the front of the draft rows in every layer's K and V
// cache, and the new lengths are written.
//
//   row(base + j) <- row(base + path[j]),  j < path_len,  base = T - n
//
// In place: path rises strictly, so path[j] >= j, and a 16-byte column of a
// (layer, K or V, sequence, KV head) is moved by one thread, which reads 8
// rows before it writes them; the rows it reads later lie at or behind every
// row it has written.  One launch for all layers; bound by its latency: 32
// layers of one sequence take 3.0 us on a B200, of 16 sequences (22 MB moved)
// 3.0 to 3.4.
#include "common.cuh"
#include "internal.h"
#include "multi.h"

namespace tb {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPath = 1024;

template <int D>
__global__ void __launch_bounds__(kThreads)
tree_accept_kernel(const uint64_t *__restrict__ caches, const int32_t *__restrict__ q_begin,
                   const int32_t *__restrict__ ctx_len, const int32_t *__restrict__ path, int path_cap,
                   const int32_t *__restrict__ path_len, int32_t *__restrict__ new_len, int Hkv, int cap,
                   uint32_t *__restrict__ flags) {
    constexpr int V16 = D / 8;
    constexpr int kBatch = 8;
    __shared__ int s_path[kMaxPath];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.y, cache = blockIdx.x, tid = threadIdx.x;
    const int T = ctx_len[b], n = q_begin[b + 1] - q_begin[b], len = path_len[b];
    // (an idle sequence's length may be anything: it comes back as it is)
    const bool idle = n == 0 && len == 0;
    bool bad = !idle && (n < 0 || n > T || T > cap || T < 0 || len < 0 || len > n || len > path_cap);
    if (!bad) {
        const int32_t *pb = path + (size_t)b * path_cap;
        for (int j = tid; j < len; j += kThreads) {
            const int v = pb[j];
            s_path[j] = v;
            bad |= v >= n || v < 0 || (j > 0 && pb[j - 1] >= v);
        }
    }
    // a cache listed again is moved once, by the block of its first entry (the
    // first entry of all is nobody's repeat, so `bad` stays what the path says)
    const uint64_t base = caches[cache];
    for (int j = tid; j < cache; j += kThreads) bad |= caches[j] == base;
    bad = __syncthreads_or(bad);
    if (tid == 0 && cache == 0) {
        if (bad) raise_flag(flags, TB_FLAG_BAD_PATH);
        new_len[b] = bad ? T : T - n + len;
    }
    if (bad) return;
    if (base == 0 || (base & 15u) != 0) {
        if (tid == 0) raise_flag(flags, TB_FLAG_BAD_CACHE);
        return;
    }
    // the leading entries that stay where they are need no move
    int j0 = 0;
    while (j0 < len && s_path[j0] == j0) ++j0;
    if (j0 == len) return;
    for (int i = tid; i < Hkv * V16; i += kThreads) {
        const int g = i / V16, c = i % V16;
        uint4 *row0 = reinterpret_cast<uint4 *>(base) + (((size_t)b * Hkv + g) * cap + (T - n)) * V16 + c;
        for (int j = j0; j < len; j += kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (j + k < len) v[k] = row0[(size_t)s_path[j + k] * V16];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (j + k < len) row0[(size_t)(j + k) * V16] = v[k];
        }
    }
}

}  // namespace

cudaError_t launch_tree_accept(const tb_dims &d, int32_t n_layers, const uint64_t *caches, const int32_t *q_begin,
                               const int32_t *ctx_len, const int32_t *path, int32_t path_cap, const int32_t *path_len,
                               int32_t *new_len, void *ws, cudaStream_t st) {
    uint32_t *flags = static_cast<uint32_t *>(ws);
    const dim3 grid(2u * (unsigned)n_layers, (unsigned)d.batch);
    if (d.head_dim == 128)
        return launch_pdl(tree_accept_kernel<128>, grid, dim3(kThreads), 0, st, caches, q_begin, ctx_len, path,
                          path_cap, path_len, new_len, d.n_kv_heads, d.ctx_cap, flags);
    return launch_pdl(tree_accept_kernel<64>, grid, dim3(kThreads), 0, st, caches, q_begin, ctx_len, path, path_cap,
                      path_len, new_len, d.n_kv_heads, d.ctx_cap, flags);
}

}  // namespace tb
