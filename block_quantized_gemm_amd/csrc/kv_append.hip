// kv_append.hip -- rows of keys and values into the pages of a cache.
//
// A key row is copied; a value row goes into the transposed blocks of 32
// tokens, so its channels land 64 bytes apart.  One thread per 8 channels of
// one row of one head: a 16-byte load of each, a 16-byte store of the key and
// eight 2-byte stores of the value.
#include "tree_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kThreads = 256;

struct KArgs {
    const uint16_t *k, *v;
    uint16_t *k_cache, *v_cache;
    const int32_t *page_table, *ctx_len, *path, *count;
    int32_t *len_out;
    int64_t k_stride, v_stride;
    int batch, n, kv_heads, dim, page_size, n_pages, max_pages;
};

__global__ __launch_bounds__(kThreads) void kv_append_rows(KArgs a, int64_t items) {
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (a.len_out && at < a.batch) {
        const int cap = a.max_pages * a.page_size;
        const int ctx = min(max(a.ctx_len[at], 0), cap);
        const int cnt = a.count ? min(max(a.count[at], 0), a.n) : a.n;
        a.len_out[at] = min(ctx + cnt, cap);
    }
    if (at >= items)
        return;
    const int pieces = a.kv_heads * a.dim / 8;
    const int c = (int)(at % pieces);
    int64_t rest = at / pieces;
    const int i = (int)(rest % a.n);
    rest /= a.n;
    const int b = (int)(rest % a.batch), layer = (int)(rest / a.batch);
    const int cnt = a.count ? min(max(a.count[b], 0), a.n) : a.n;
    const int cap = a.max_pages * a.page_size;
    const int pos = min(max(a.ctx_len[b], 0), cap) + i;
    const int src = a.path ? a.path[(int64_t)b * a.n + i] : i;
    if (i >= cnt || pos >= cap || src < 0 || src >= a.n)
        return;
    const int page = a.page_table[(int64_t)b * a.max_pages + pos / a.page_size];
    if (page < 0 || page >= a.n_pages)
        return;
    const int off = pos % a.page_size, h = c * 8 / a.dim, d = c * 8 % a.dim;
    const int64_t row = ((int64_t)layer * a.batch + b) * a.n + src;
    const int64_t base = (((int64_t)layer * a.n_pages + page) * a.kv_heads + h) * a.page_size * a.dim;
    const u32x4 kx = ld16(a.k + row * a.k_stride + c * 8), vx = ld16(a.v + row * a.v_stride + c * 8);
    *reinterpret_cast<u32x4 *>(a.k_cache + base + (int64_t)off * a.dim + d) = kx;
    uint16_t *vp = a.v_cache + base + (int64_t)(off / kVBlock) * kVBlock * a.dim + off % kVBlock;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        vp[(d + e) * kVBlock] = (uint16_t)(vx[e >> 1] >> (16 * (e & 1)));
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &p) {
    KArgs a{static_cast<const uint16_t *>(p.k), static_cast<const uint16_t *>(p.v),
            static_cast<uint16_t *>(p.k_cache), static_cast<uint16_t *>(p.v_cache), p.page_table, p.ctx_len, p.path,
            p.count, p.len_out, p.k_stride, p.v_stride, p.batch, p.n, p.kv_heads, p.head_dim, p.page_size,
            p.n_pages, p.max_pages};
    const int64_t items = (int64_t)p.n_layers * p.batch * p.n * (p.kv_heads * p.head_dim / 8);
    const int64_t groups = (std::max<int64_t>(items, p.batch) + kThreads - 1) / kThreads;
    if (groups > 0x7FFFFFFF)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(kv_append_rows, dim3((unsigned)groups), dim3(kThreads), 0, p.stream, a, items);
    return hipGetLastError();
}

}  // namespace vq
