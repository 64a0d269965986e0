// tree_internal.h -- host-side declarations of the speculative-step operators
// (tree attention, tree acceptance, cache append).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "vq.h"

namespace vq {

// Tokens per transposed block of the value cache: the depth of one 16-bit MFMA.
constexpr int kVBlock = 32;

// Arguments of one tree attention launch, already checked.
struct TreeAttnArgs {
    const void *q, *k, *v;
    int q_stride, k_stride, v_stride;  // elements between rows
    int dtype;
    const void *k_cache, *v_cache;
    const int32_t *page_table, *ctx_len;
    const uint64_t *tree_mask;  // or null: a chain
    const int32_t *n_nodes;     // or null: n
    void *out;
    int batch, n, q_heads, kv_heads, head_dim;
    int page_size, n_pages, max_pages;
    float scale;
    void *workspace;
    hipStream_t stream;
};
hipError_t launch_tree_attention(const TreeAttnArgs &a);
size_t tree_attention_workspace(int batch, int n, int q_heads, int kv_heads, int head_dim);

// Arguments of one tree acceptance, already checked.
struct TreeVerifyArgs {
    const void *target, *draft;  // draft null: children were given, not drawn
    int dtype;
    const int32_t *node_tokens, *parents, *n_nodes;
    const float *temperature, *uniforms, *noise;
    int32_t *tokens_out, *path_out, *count_out;
    int batch, n, vocab;
    void *workspace;
    hipStream_t stream;
};
hipError_t launch_tree_verify(const TreeVerifyArgs &a);
size_t tree_verify_workspace(int batch, int n, int vocab);

// Arguments of one cache append, already checked.
struct KvAppendArgs {
    const void *k, *v;
    int k_stride, v_stride;
    void *k_cache, *v_cache;
    const int32_t *page_table, *ctx_len, *path, *count;
    int32_t *len_out;
    int n_layers, batch, n, kv_heads, head_dim;
    int page_size, n_pages, max_pages;
    hipStream_t stream;
};
hipError_t launch_kv_append(const KvAppendArgs &a);
// Whether one launch can cover this many rows (a grid dimension holds 2^32 - 1
// threads, and a launch past that is refused only when it is made).
bool kv_append_fits(int64_t n_layers, int64_t batch, int64_t n, int64_t kv_heads, int64_t head_dim);

}  // namespace vq
