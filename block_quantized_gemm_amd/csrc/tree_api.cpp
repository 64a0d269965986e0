// tree_api.cpp -- the C ABI of the speculative-step operators: argument
// validation and dispatch, under the conventions of vq.h (every argument is
// checked before the first HIP call; on any error nothing is enqueued).
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "tree_internal.h"
#include "vq.h"

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

int check_device() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0)
        return VQ_ERR_DEVICE;
    const int known = dev < kMaxDevices ? g_dev_ok[dev].load(std::memory_order_relaxed) : 0;
    if (known)
        return known == 1 ? VQ_OK : VQ_ERR_DEVICE;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return VQ_ERR_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < kMaxDevices)
        g_dev_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? VQ_OK : VQ_ERR_DEVICE;
}

bool all_aligned(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15u)
            return false;
    return true;
}
bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool half_type(int d) { return d == VQ_DTYPE_F16 || d == VQ_DTYPE_BF16; }
bool stride_ok(int64_t s, int64_t width) { return s % 8 == 0 && in(s, width, VQ_MAX_DIM); }

bool heads_ok(int64_t batch, int64_t kv_heads, int64_t head_dim) {
    return in(batch, 1, VQ_MAX_BATCH) && in(kv_heads, 1, VQ_MAX_HEADS) &&
           (head_dim == 64 || head_dim == 128 || head_dim == 256);
}
bool cache_ok(int64_t page_size, int64_t n_pages, int64_t max_pages) {
    return (page_size == 32 || page_size == 64 || page_size == 128 || page_size == 256) &&
           in(n_pages, 1, VQ_MAX_DIM) && in(max_pages, 1, ((int64_t)1 << 30) / page_size);
}
bool attn_ok(int64_t batch, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    return heads_ok(batch, kv_heads, head_dim) && in(n, 1, VQ_MAX_TREE_NODES) && in(q_heads, 1, VQ_MAX_HEADS) &&
           q_heads % kv_heads == 0;
}
bool verify_ok(int64_t batch, int64_t n, int64_t vocab) {
    return in(batch, 1, VQ_MAX_BATCH) && in(n, 1, VQ_MAX_TREE_NODES) && in(vocab, 1, VQ_MAX_DIM);
}
int status(hipError_t e) { return e == hipSuccess ? VQ_OK : VQ_ERR_LAUNCH; }

}  // namespace

extern "C" {

size_t vq_tree_attention_workspace_bytes(int64_t batch, int64_t n, int64_t q_heads, int64_t kv_heads,
                                         int64_t head_dim) {
    if (!attn_ok(batch, n, q_heads, kv_heads, head_dim))
        return 0;
    return vq::tree_attention_workspace((int)batch, (int)n, (int)q_heads, (int)kv_heads, (int)head_dim);
}

int vq_tree_attention(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                      int64_t v_stride, int dtype, const void *k_cache, const void *v_cache,
                      const int32_t *page_table, const int32_t *ctx_len, const uint64_t *tree_mask,
                      const int32_t *n_nodes, void *out, int64_t batch, int64_t n, int64_t q_heads,
                      int64_t kv_heads, int64_t head_dim, int64_t page_size, int64_t n_pages, int64_t max_pages,
                      float scale, void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k || !v || !k_cache || !v_cache || !page_table || !ctx_len || !out)
        return VQ_ERR_NULL_POINTER;
    if (!half_type(dtype))
        return VQ_ERR_BAD_DTYPE;
    if (!attn_ok(batch, n, q_heads, kv_heads, head_dim) || !cache_ok(page_size, n_pages, max_pages) ||
        !stride_ok(q_stride, q_heads * head_dim) || !stride_ok(k_stride, kv_heads * head_dim) ||
        !stride_ok(v_stride, kv_heads * head_dim))
        return VQ_ERR_BAD_SHAPE;
    if (!all_aligned({q, k, v, k_cache, v_cache, page_table, ctx_len, tree_mask, n_nodes, out, workspace}))
        return VQ_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < vq::tree_attention_workspace((int)batch, (int)n, (int)q_heads,
                                                                     (int)kv_heads, (int)head_dim))
        return VQ_ERR_WORKSPACE;
    const int dev = check_device();
    if (dev != VQ_OK)
        return dev;
    vq::TreeAttnArgs a{q, k, v, (int)q_stride, (int)k_stride, (int)v_stride, dtype, k_cache, v_cache, page_table,
                       ctx_len, tree_mask, n_nodes, out, (int)batch, (int)n, (int)q_heads, (int)kv_heads,
                       (int)head_dim, (int)page_size, (int)n_pages, (int)max_pages, scale, workspace,
                       static_cast<hipStream_t>(stream)};
    return status(vq::launch_tree_attention(a));
}

size_t vq_tree_verify_workspace_bytes(int64_t batch, int64_t n, int64_t vocab) {
    if (!verify_ok(batch, n, vocab))
        return 0;
    return vq::tree_verify_workspace((int)batch, (int)n, (int)vocab);
}

int vq_tree_verify(const void *target, const void *draft, int logits_dtype, const int32_t *node_tokens,
                   const int32_t *parents, const int32_t *n_nodes, const float *temperature,
                   const float *uniforms, const float *noise, int32_t *tokens_out, int32_t *path_out,
                   int32_t *count_out, int64_t batch, int64_t n, int64_t vocab, void *workspace,
                   size_t workspace_bytes, void *stream) {
    if (!target || !node_tokens || !uniforms || !noise || !tokens_out || !path_out || !count_out)
        return VQ_ERR_NULL_POINTER;
    if (logits_dtype != VQ_DTYPE_F32 && !half_type(logits_dtype))
        return VQ_ERR_BAD_DTYPE;
    if (!verify_ok(batch, n, vocab))
        return VQ_ERR_BAD_SHAPE;
    if (!all_aligned({target, draft, node_tokens, parents, n_nodes, temperature, uniforms, noise, tokens_out,
                      path_out, count_out, workspace}))
        return VQ_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < vq::tree_verify_workspace((int)batch, (int)n, (int)vocab))
        return VQ_ERR_WORKSPACE;
    const int dev = check_device();
    if (dev != VQ_OK)
        return dev;
    vq::TreeVerifyArgs a{target, draft, logits_dtype, node_tokens, parents, n_nodes, temperature, uniforms, noise,
                         tokens_out, path_out, count_out, (int)batch, (int)n, (int)vocab, workspace,
                         static_cast<hipStream_t>(stream)};
    return status(vq::launch_tree_verify(a));
}

int vq_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int dtype, void *k_cache,
                 void *v_cache, const int32_t *page_table, const int32_t *ctx_len, const int32_t *path,
                 const int32_t *count, int32_t *len_out, int64_t n_layers, int64_t batch, int64_t n,
                 int64_t kv_heads, int64_t head_dim, int64_t page_size, int64_t n_pages, int64_t max_pages,
                 void *stream) {
    if (!k || !v || !k_cache || !v_cache || !page_table || !ctx_len)
        return VQ_ERR_NULL_POINTER;
    if (!half_type(dtype))
        return VQ_ERR_BAD_DTYPE;
    if (!heads_ok(batch, kv_heads, head_dim) || !cache_ok(page_size, n_pages, max_pages) ||
        !in(n_layers, 1, VQ_MAX_HEADS) || !in(n, 1, VQ_MAX_DIM) || !stride_ok(k_stride, kv_heads * head_dim) ||
        !stride_ok(v_stride, kv_heads * head_dim) || !vq::kv_append_fits(n_layers, batch, n, kv_heads, head_dim))
        return VQ_ERR_BAD_SHAPE;
    if (!all_aligned({k, v, k_cache, v_cache, page_table, ctx_len, path, count, len_out}))
        return VQ_ERR_MISALIGNED;
    const int dev = check_device();
    if (dev != VQ_OK)
        return dev;
    vq::KvAppendArgs a{k, v, (int)k_stride, (int)v_stride, k_cache, v_cache, page_table, ctx_len, path, count,
                       len_out, (int)n_layers, (int)batch, (int)n, (int)kv_heads, (int)head_dim, (int)page_size,
                       (int)n_pages, (int)max_pages, static_cast<hipStream_t>(stream)};
    return status(vq::launch_kv_append(a));
}

}  // extern "C"
