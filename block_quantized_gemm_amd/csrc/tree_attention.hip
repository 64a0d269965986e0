// tree_attention.hip -- attention of a tree of drafted tokens over a paged cache.
//
// For each query row (node i of sequence b, query head h):
//   out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  s_t = scale * (q . k_t),
// over the cached positions t < ctx_len[b] and the nodes its mask names, in
// one pass with a running maximum m and sum: when m grows, what was summed is
// multiplied by exp(m_old - m_new).
//
// One workgroup per query row, 256 positions at a time: a thread per position
// forms its score, the workgroup the new maximum, then a thread per channel
// adds the 256 weighted values.
#include "tree_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kThreads = 256;

struct KArgs {
    const uint16_t *q, *k, *v, *k_cache, *v_cache;
    const int32_t *page_table, *ctx_len;
    const uint64_t *tree_mask;
    const int32_t *n_nodes;
    uint16_t *out;
    int64_t q_stride, k_stride, v_stride;
    int n, q_heads, kv_heads, dim, page_size, n_pages, max_pages;
    float scale;
};

template <int DT>
__device__ __forceinline__ float to_f32(uint16_t h) {
    if constexpr (DT == VQ_DTYPE_BF16)
        return __builtin_bit_cast(float, (uint32_t)h << 16);
    else
        return static_cast<float>(__builtin_bit_cast(_Float16, h));
}

// Workgroup maximum or sum; every thread gets it.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float x, float *red) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const float o = __shfl_xor(x, off, 64);
        x = MAX ? fmaxf(x, o) : x + o;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w)
        x = MAX ? fmaxf(x, red[w]) : x + red[w];
    return x;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void tree_attention_rows(KArgs a) {
    __shared__ float qs[256], ps[kThreads], red[kThreads / 64];
    const int tid = (int)threadIdx.x;
    const int h = (int)blockIdx.x % a.q_heads, row = (int)blockIdx.x / a.q_heads;
    const int b = row / a.n, i = row - b * a.n;
    const int hk = h / (a.q_heads / a.kv_heads);
    const int ctx = min(max(a.ctx_len[b], 0), a.max_pages * a.page_size);
    const int nodes = a.n_nodes ? min(max(a.n_nodes[b], 0), a.n) : a.n;
    uint64_t mask = a.tree_mask ? a.tree_mask[row] : ~0ull >> (63 - i);
    mask &= nodes == 0 ? 0 : ~0ull >> (64 - nodes);
    uint16_t *out = a.out + ((int64_t)row * a.q_heads + h) * a.dim;
    const bool live = i < nodes && (ctx > 0 || mask);
    if (!live) {
        if (tid < a.dim)
            out[tid] = 0;
        return;
    }
    if (tid < a.dim)
        qs[tid] = to_f32<DT>(a.q[row * a.q_stride + (int64_t)h * a.dim + tid]);
    __syncthreads();
    float m = -INFINITY, total = 0.f, acc = 0.f;
    for (int t0 = 0; t0 < ctx + nodes; t0 += kThreads) {
        const int t = t0 + tid;
        float s = -INFINITY;
        if (t < ctx || (t < ctx + nodes && (mask >> (t - ctx) & 1))) {
            const uint16_t *kr = nullptr;
            if (t >= ctx) {
                kr = a.k + ((int64_t)b * a.n + (t - ctx)) * a.k_stride + (int64_t)hk * a.dim;
            } else {
                const int page = a.page_table[(int64_t)b * a.max_pages + t / a.page_size];
                if (page >= 0 && page < a.n_pages)
                    kr = a.k_cache + (((int64_t)page * a.kv_heads + hk) * a.page_size + t % a.page_size) * a.dim;
            }
            s = 0.f;
            if (kr)
                for (int d = 0; d < a.dim; ++d)
                    s += qs[d] * to_f32<DT>(kr[d]);
            s *= a.scale;
        }
        const float m_new = fmaxf(m, block_reduce<true>(s, red));
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const bool see = t < ctx || (t < ctx + nodes && (mask >> (t - ctx) & 1));
        const float p = see ? expf(s - base) : 0.f;
        const float shrink = expf(m - base);
        ps[tid] = p;
        total = total * shrink + block_reduce<false>(p, red);  // its barriers also publish ps
        m = m_new;
        if (tid < a.dim) {
            acc *= shrink;
            const int end = min(kThreads, ctx + nodes - t0);
            for (int e = 0; e < end; ++e) {
                const int u = t0 + e;
                if (u >= ctx) {
                    if (mask >> (u - ctx) & 1)
                        acc += ps[e] * to_f32<DT>(a.v[((int64_t)b * a.n + (u - ctx)) * a.v_stride +
                                                      (int64_t)hk * a.dim + tid]);
                    continue;
                }
                const int page = a.page_table[(int64_t)b * a.max_pages + u / a.page_size];
                if (page >= 0 && page < a.n_pages) {
                    const int off = u % a.page_size;
                    acc += ps[e] * to_f32<DT>(a.v_cache[(((int64_t)page * a.kv_heads + hk) * a.page_size +
                                                         (off / kVBlock) * kVBlock) * a.dim +
                                                        tid * kVBlock + off % kVBlock]);
                }
            }
        }
        __syncthreads();
    }
    if (tid < a.dim)
        store_out(out, DT, tid, acc / total);
}

}  // namespace

size_t tree_attention_workspace(int, int, int, int, int) { return 16; }

hipError_t launch_tree_attention(const TreeAttnArgs &p) {
    KArgs a{static_cast<const uint16_t *>(p.q), static_cast<const uint16_t *>(p.k),
            static_cast<const uint16_t *>(p.v), static_cast<const uint16_t *>(p.k_cache),
            static_cast<const uint16_t *>(p.v_cache), p.page_table, p.ctx_len, p.tree_mask, p.n_nodes,
            static_cast<uint16_t *>(p.out), p.q_stride, p.k_stride, p.v_stride, p.n, p.q_heads, p.kv_heads,
            p.head_dim, p.page_size, p.n_pages, p.max_pages, p.scale};
    const dim3 grid((unsigned)p.batch * p.n * p.q_heads);
    if (p.dtype == VQ_DTYPE_BF16)
        hipLaunchKernelGGL(tree_attention_rows<VQ_DTYPE_BF16>, grid, dim3(kThreads), 0, p.stream, a);
    else
        hipLaunchKernelGGL(tree_attention_rows<VQ_DTYPE_F16>, grid, dim3(kThreads), 0, p.stream, a);
    return hipGetLastError();
}

}  // namespace vq
