// tree_verify.hip -- acceptance of a tree of drafted tokens from given random
// numbers, so that the committed tokens follow the target's distribution.
//
// At a node with target p and drafter q the children are tried in turn; each
// rejection replaces p by the normalised positive part of p - q.  Unnormalised,
//   r_j = max(0, max(0, ... max(0, p - s_0 q) ... ) - s_(j-1) q)
//       = max(0, p - S_j q),  S_j = s_0 + ... + s_(j-1),  s_j = sum r_j,
// because max(0, max(0, a - b) - c) = max(0, a - b - c) for b, c >= 0: one
// scalar carries everything that earlier rejections did.  The last token is
// argmax r / e with exponential variates e: min over x of e_x / r_x is at x
// with probability r_x / sum r, so no running sum over the vocabulary is
// compared with a threshold, and the result does not hang on its rounding.
//
// Two kernels: the first reads every row once for its maximum and sum of
// exponentials, one workgroup per row; the second, one workgroup per
// sequence, walks the tree and draws the last token.
#include "tree_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kStatThreads = 256;
constexpr int kWalkThreads = 1024;

struct KArgs {
    const void *target, *draft;
    const int32_t *node_tokens, *parents, *n_nodes;
    const float *temperature, *uniforms, *noise;
    int32_t *tokens_out, *path_out, *count_out;
    int n, vocab;
};

// What the first kernel leaves of a row: softmax maximum and 1 / sum, and the
// greedy choice.
struct RowStat {
    float m, inv, mq, invq;
    int32_t best;
    int32_t pad[3];
};

template <int DT>
__device__ __forceinline__ float logit_at(const void *p, int64_t i) {
    if constexpr (DT == VQ_DTYPE_F32)
        return static_cast<const float *>(p)[i];
    else if constexpr (DT == VQ_DTYPE_BF16)
        return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    else
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<const uint16_t *>(p)[i]));
}

// Order-preserving key of a float and its index: larger values first, NaN
// before all, -0 as +0, the lower index of equal values.
__device__ __forceinline__ uint64_t key_of(float x, int idx) {
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    if (u == 0x80000000u)
        u = 0u;
    u = x != x ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)u << 32) | (uint32_t)~(uint32_t)idx;
}

struct MaxOp {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; }
};
struct SumOp {
    __device__ float operator()(float a, float b) const { return a + b; }
};

__device__ __forceinline__ float lane_xor(float x, int off) { return __shfl_xor(x, off, 64); }
__device__ __forceinline__ uint64_t lane_xor(uint64_t x, int off) {
    const uint32_t lo = __shfl_xor((uint32_t)x, off, 64), hi = __shfl_xor((uint32_t)(x >> 32), off, 64);
    return ((uint64_t)hi << 32) | lo;
}

// Reduction over a workgroup of THREADS; every thread gets it.
template <int THREADS, typename Op, typename T>
__device__ __forceinline__ T block_reduce(T x, Op op, uint64_t *red64) {
    T *red = reinterpret_cast<T *>(red64);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        x = op(x, lane_xor(x, off));
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w)
        x = op(x, red[w]);
    return x;
}

__device__ __forceinline__ int live_nodes(const KArgs &a, int b) {
    return a.n_nodes ? min(max(a.n_nodes[b], 0), a.n) : a.n;
}
__device__ __forceinline__ int parent_of(const KArgs &a, int b, int i) {
    return a.parents ? a.parents[(int64_t)b * a.n + i] : i - 1;
}
// log2(e) / T: exp((l - m) / T) = exp2((l - m) * c); a greedy sequence's
// probabilities are not used
__device__ __forceinline__ float exponent_scale(const KArgs &a, int b) {
    const float t = a.temperature ? a.temperature[b] : 1.f;
    return t > 0.f ? 1.44269504088896f / t : 0.f;
}

template <int DT>
__device__ __forceinline__ void softmax_stats(const void *row, int vocab, float c, uint64_t *red, float &m,
                                              float &inv) {
    float mx = -INFINITY;
    for (int x = (int)threadIdx.x; x < vocab; x += kStatThreads)
        mx = fmaxf(mx, logit_at<DT>(row, x));
    m = block_reduce<kStatThreads>(mx, MaxOp{}, red);
    float sum = 0.f;
    for (int x = (int)threadIdx.x; x < vocab; x += kStatThreads)
        sum += exp2f((logit_at<DT>(row, x) - m) * c);
    inv = 1.f / block_reduce<kStatThreads>(sum, SumOp{}, red);
}

template <int DT>
__device__ __forceinline__ const void *row_ptr(const void *base, const KArgs &a, int b, int v) {
    constexpr int kElem = DT == VQ_DTYPE_F32 ? 4 : 2;
    return static_cast<const char *>(base) + ((int64_t)b * a.n + v) * a.vocab * kElem;
}

template <int DT>
__global__ __launch_bounds__(kStatThreads) void tree_row_stats(KArgs a, RowStat *stats) {
    __shared__ uint64_t red[kStatThreads / 64];
    const int v = (int)blockIdx.x, b = (int)blockIdx.y, nodes = live_nodes(a, b);
    if (v >= nodes)
        return;
    const float c = exponent_scale(a, b);
    RowStat st{};
    const void *row = row_ptr<DT>(a.target, a, b, v);
    if (c == 0.f) {
        uint64_t best = 0;
        for (int x = (int)threadIdx.x; x < a.vocab; x += kStatThreads) {
            const uint64_t k = key_of(logit_at<DT>(row, x), x);
            best = k > best ? k : best;
        }
        st.best = (int32_t)~(uint32_t)block_reduce<kStatThreads>(best, MaxOp{}, red);
    } else {
        softmax_stats<DT>(row, a.vocab, c, red, st.m, st.inv);
        bool inner = false;
        for (int i = v + 1; i < nodes; ++i)
            inner = inner || parent_of(a, b, i) == v;
        if (a.draft && inner)
            softmax_stats<DT>(row_ptr<DT>(a.draft, a, b, v), a.vocab, c, red, st.mq, st.invq);
    }
    if (threadIdx.x == 0)
        stats[(int64_t)b * a.n + v] = st;
}

template <int DT>
__global__ __launch_bounds__(kWalkThreads) void tree_walk(KArgs a, const RowStat *stats) {
    __shared__ uint64_t red[kWalkThreads / 64];
    __shared__ int32_t gone[VQ_MAX_TREE_NODES];  // tokens of the rejected children (no draft logits)
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x, nodes = live_nodes(a, b);
    int32_t *tokens = a.tokens_out + (int64_t)b * a.n, *path = a.path_out + (int64_t)b * a.n;
    const int32_t *drafted = a.node_tokens + (int64_t)b * a.n;
    const float *noise = a.noise + (int64_t)b * a.vocab;
    if (tid < a.n) {
        tokens[tid] = -1;
        path[tid] = -1;
    }
    if (nodes == 0) {
        if (tid == 0)
            a.count_out[b] = 0;
        return;
    }
    __syncthreads();
    const float c = exponent_scale(a, b);
    int v = 0, count = 1;
    if (tid == 0)
        path[0] = 0;
    for (;;) {
        const RowStat st = stats[(int64_t)b * a.n + v];
        const void *rp = row_ptr<DT>(a.target, a, b, v);
        const void *rq = a.draft ? row_ptr<DT>(a.draft, a, b, v) : nullptr;
        auto prob = [&](int x) { return exp2f((logit_at<DT>(rp, x) - st.m) * c) * st.inv; };
        auto drawn = [&](int x) { return exp2f((logit_at<DT>(rq, x) - st.mq) * c) * st.invq; };
        float S = 0.f, s = 1.f;
        int n_gone = 0, next = -1;
        bool stale = false;  // s is older than S
        auto left = [&](int x) -> float {
            const float p = prob(x);
            if (rq)
                return S > 0.f ? fmaxf(0.f, p - S * drawn(x)) : p;
            for (int g = 0; g < n_gone; ++g)
                if (gone[g] == x)
                    return 0.f;
            return p;
        };
        for (int kid = v + 1; kid < nodes && next < 0; ++kid) {
            if (parent_of(a, b, kid) != v)
                continue;
            const int x = drafted[kid];
            if (c == 0.f) {
                next = x == st.best ? kid : -1;
                continue;
            }
            if (stale) {
                float sum = 0.f;
                for (int y = tid; y < a.vocab; y += kWalkThreads)
                    sum += left(y);
                s = block_reduce<kWalkThreads>(sum, SumOp{}, red);
                stale = false;
            }
            const bool inside = x >= 0 && x < a.vocab;
            const float rx = inside ? left(x) : 0.f;
            const float qx = rq ? (inside ? drawn(x) : 0.f) : 1.f;
            if (inside && a.uniforms[(int64_t)b * a.n + kid] * qx * s < rx) {
                next = kid;
                continue;
            }
            if (rq) {
                S += s;
                stale = true;
            } else {
                s -= rx;
                __syncthreads();
                if (tid == 0)
                    gone[n_gone] = x;
                ++n_gone;
                __syncthreads();
            }
        }
        if (next >= 0) {
            if (tid == 0) {
                tokens[count - 1] = drafted[next];
                path[count] = next;
            }
            ++count;
            v = next;
            continue;
        }
        int32_t last = st.best;
        if (c != 0.f) {
            uint64_t best = 0;
            for (int pass = 0; pass < 2 && best == 0; ++pass) {
                for (int x = tid; x < a.vocab; x += kWalkThreads) {
                    const float r = pass == 0 ? left(x) : prob(x);
                    if (r > 0.f) {
                        const uint64_t k = key_of(r / noise[x], x);
                        best = k > best ? k : best;
                    }
                }
                best = block_reduce<kWalkThreads>(best, MaxOp{}, red);
            }
            last = best ? (int32_t)~(uint32_t)best : 0;
        }
        if (tid == 0) {
            tokens[count - 1] = last;
            a.count_out[b] = count;
        }
        return;
    }
}

template <int DT>
void launch_dt(const KArgs &a, int batch, void *workspace, hipStream_t stream) {
    RowStat *stats = static_cast<RowStat *>(workspace);
    hipLaunchKernelGGL(tree_row_stats<DT>, dim3(a.n, batch), dim3(kStatThreads), 0, stream, a, stats);
    hipLaunchKernelGGL(tree_walk<DT>, dim3(batch), dim3(kWalkThreads), 0, stream, a, stats);
}

}  // namespace

size_t tree_verify_workspace(int batch, int n, int) { return (size_t)batch * n * sizeof(RowStat); }

hipError_t launch_tree_verify(const TreeVerifyArgs &p) {
    KArgs a{p.target, p.draft, p.node_tokens, p.parents, p.n_nodes, p.temperature, p.uniforms, p.noise,
            p.tokens_out, p.path_out, p.count_out, p.n, p.vocab};
    if (p.dtype == VQ_DTYPE_F32)
        launch_dt<VQ_DTYPE_F32>(a, p.batch, p.workspace, p.stream);
    else if (p.dtype == VQ_DTYPE_BF16)
        launch_dt<VQ_DTYPE_BF16>(a, p.batch, p.workspace, p.stream);
    else
        launch_dt<VQ_DTYPE_F16>(a, p.batch, p.workspace, p.stream);
    return hipGetLastError();
}

}  // namespace vq
