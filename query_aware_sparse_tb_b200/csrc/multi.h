// Launchers of the calls that take several new tokens of a sequence at once
// (not part of the ABI): norms and rotation with the cache write (rope.cu),
// prompt and tree attention (multi_attn.cu), tree acceptance (tree.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tb.h"

namespace tb {

// ---- prompt and tree attention (multi_attn.cu) ----
size_t multi_attn_ws_bytes(const tb_dims &d, int32_t n_tokens, int32_t max_new, bool tree);
// mask == nullptr: causal; else the tree's attention bits [n_tokens][ceil(max_new/32)].
cudaError_t launch_multi_attn(const tb_dims &d, const uint16_t *Q, const uint16_t *K, const uint16_t *V,
                              const int32_t *q_begin, int32_t n_tokens, int32_t max_new, const int32_t *ctx_len,
                              const uint32_t *mask, float scale, uint16_t *out, void *ws, cudaStream_t st);

// ---- norms, rotation, cache write (rope.cu) ----
cudaError_t launch_norm_rope_append(const tb_dims &d, const uint16_t *qkv, int64_t row_stride, const int32_t *q_begin,
                                    int32_t n_tokens, const int32_t *ctx_len, const int32_t *pos, const uint16_t *qw,
                                    const uint16_t *kw, float eps, const double *inv_freq, int32_t rot_dim,
                                    int32_t style, uint16_t *Q, uint16_t *K, uint16_t *V, void *ws, cudaStream_t st);

// ---- tree acceptance (tree.cu) ----
cudaError_t launch_tree_accept(const tb_dims &d, int32_t n_layers, const uint64_t *caches, const int32_t *q_begin,
                               const int32_t *ctx_len, const int32_t *path, int32_t path_cap,
                               const int32_t *path_len, int32_t *new_len, void *ws, cudaStream_t st);

// ---- where a packed token lies ----
// Tokens of sequence b are q_begin[b] .. q_begin[b+1] of the packed arrays; a
// q_begin that runs backwards or outside [0, n_tokens] is clamped, so no index
// derived from it leaves the arrays.
struct SeqSpan {
    int begin, n;
};
__device__ __forceinline__ SeqSpan seq_span(const int32_t *q_begin, int b, int n_tokens) {
    const int s0 = min(max(q_begin[b], 0), n_tokens);
    const int s1 = min(max(q_begin[b + 1], s0), n_tokens);
    return {s0, s1 - s0};
}

}  // namespace tb
