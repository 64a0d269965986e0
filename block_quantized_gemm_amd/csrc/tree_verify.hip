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
// Three kernels.  The first reads every row once, a workgroup per chunk of 8192
// logits held in registers, and leaves each chunk's maximum and sum of
// exponentials (or, for a greedy sequence, its best key).  The second, one
// workgroup per sequence, joins the chunks, looks the drafted tokens up and
// walks the tree; only a node that is tried again after a rejection costs it
// another pass over that node's two rows.  The third draws the last token,
// the row split over many workgroups; the last to arrive writes it.
//
// Measured on one MI355X: the whole call, and each kernel's median in a trace,
// whose own overhead is in it:
//                                                           call          stats   walk   draw
//   1 chain of 16, 151,936 bf16 logits, drawn children      19 to 20 us     5.2    5.5    6.7
//   4 trees of up to 61, 32,001 fp32 logits, given          23 to 25        7.4    9.8    6.8
//   32 trees of up to 16, 151,936 bf16 logits, drawn        98 to 112      45.3   61.5   11.1
// The first kernel is bound by reading the rows (175 MB of the large batch's,
// 3.9 TB/s), small calls by the three kernels' start and their chains of
// dependent loads, the smallest by the host's three launches (19 us from
// Python).  A retry's pass over two rows is the work of one workgroup:
// 152k tokens cost it two exponentials each, about 20 us of one CU, and the walk
// lasts as long as its unluckiest sequence.
#include "tree_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kNodes = VQ_MAX_TREE_NODES;
constexpr int kThreads = 256;
constexpr int kWalkThreads = 1024;
constexpr int kPieces = 4;                   // pieces of 8 logits a lane holds
constexpr int kChunk = kThreads * 8 * kPieces;  // logits of a workgroup of the first kernel
constexpr int kJoinLanes = 16;               // lanes that join a row's chunks in the second
constexpr int kDrawChunk = kThreads * 8 * 2;  // tokens of a workgroup of the third

struct KArgs {
    const void *target, *draft;
    const int32_t *node_tokens, *parents, *n_nodes;
    const float *temperature, *uniforms, *noise;
    int32_t *tokens_out, *path_out, *count_out;
    uint2 *part;          // [batch][target, draft][n][chunks]
    struct Last *last;    // [batch]
    int n, vocab, chunks;
};

// What the walk leaves for the draw: the node whose row is drawn from, the
// softmax terms of its rows, the remainder's scalar S, the rejected tokens
// (without draft logits), and the draw's best key and arrivals.
struct Last {
    uint64_t key;
    uint32_t arrived;
    int32_t node, at;     // node < 0: no draw; at: the token's place in the outputs
    float m, inv, mq, invq, S;
    int32_t n_gone;
    int32_t gone[kNodes];
};

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

// Reduction over runs of LANES lanes (all of a run active); each gets it.
template <int LANES, typename Op, typename T>
__device__ __forceinline__ T wave_reduce(T x, Op op) {
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1)
        x = op(x, lane_xor(x, off));
    return x;
}

template <int DT>
__device__ __forceinline__ float logit_at(const void *p, int64_t i) {
    if constexpr (DT == VQ_DTYPE_F32)
        return static_cast<const float *>(p)[i];
    else if constexpr (DT == VQ_DTYPE_BF16)
        return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    else
        return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<const uint16_t *>(p)[i]));
}

// max(0, p - S q): one rounding, the product's is inside the fma.
__device__ __forceinline__ float left_of(float p, float S, float q) { return fmaxf(0.f, fmaf(-S, q, p)); }

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

// One row of logits, read 8 at a time from 16-byte aligned addresses: the row
// begins `shift` elements after its first piece.  Elements outside the row
// read as -inf; nothing past the row's last dword is touched.
template <int DT>
struct Row {
    static constexpr int kElem = DT == VQ_DTYPE_F32 ? 4 : 2;
    rsrc_t r;
    int shift, vocab;

    __device__ __forceinline__ Row(const void *base, const KArgs &a, int b, int v) : vocab(a.vocab) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(base) + ((uint64_t)b * a.n + v) * (uint64_t)a.vocab * kElem;
        shift = uniform((int)(at & 15) / kElem);
        r = make_rsrc(reinterpret_cast<const void *>(at & ~(uintptr_t)15),
                      (uint32_t)((shift + a.vocab) * kElem + 3) & ~3u);
    }
    static __device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

    // elements pos - shift .. + 8 of the row, pos a multiple of 8
    __device__ __forceinline__ void load(int pos, u32x4 (&raw)[kElem / 2]) const {
#pragma unroll
        for (int i = 0; i < kElem / 2; ++i)
            raw[i] = bload16<kAuxCached>(r, pos * kElem + 16 * i, 0);
    }
    __device__ __forceinline__ void values(const u32x4 (&raw)[kElem / 2], int pos, float (&x)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (DT == VQ_DTYPE_F32) {
                const uint32_t w = raw[e >> 2][e & 3];
                x[e] = __builtin_bit_cast(float, w);
            } else {
                const uint32_t w = raw[0][e >> 1], h = e & 1 ? w >> 16 : w & 0xFFFFu;
                x[e] = DT == VQ_DTYPE_BF16 ? __builtin_bit_cast(float, h << 16) : h2f(h);
            }
        }
        if (pos < shift || pos + 8 > shift + vocab)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = pos + e >= shift && pos + e < shift + vocab ? x[e] : -INFINITY;
    }
    __device__ __forceinline__ int end() const { return shift + vocab; }
};

template <int DT>
__global__ __launch_bounds__(kThreads) void tree_row_stats(KArgs a) {
    __shared__ uint64_t red[kThreads / 64];
    const int lane = (int)(threadIdx.x & 63), wave = wave_id(), chunk = (int)blockIdx.x;
    const bool draft = (int)blockIdx.y >= a.n;
    const int v = (int)blockIdx.y - (draft ? a.n : 0), b = (int)blockIdx.z, nodes = live_nodes(a, b);
    if (v >= nodes)
        return;
    const float c = exponent_scale(a, b);
    if (draft) {
        // a drafter's row counts only where it has children and is asked for probabilities
        if (c == 0.f || !__any(lane > v && lane < nodes && parent_of(a, b, lane) == v))
            return;
    }
    const Row<DT> row(draft ? a.draft : a.target, a, b, v);
    u32x4 raw[kPieces][Row<DT>::kElem / 2];
    const int pos0 = chunk * kChunk + (int)threadIdx.x * 8;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        row.load(pos0 + i * kThreads * 8, raw[i]);
    uint2 *out = a.part + (((int64_t)b * 2 + (draft ? 1 : 0)) * a.n + v) * a.chunks + chunk;
    float x[8];
    if (c == 0.f) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int pos = pos0 + i * kThreads * 8;
            row.values(raw[i], pos, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t k = key_of(x[e], pos + e - row.shift);
                if (pos + e >= row.shift && pos + e < row.end())
                    best = k > best ? k : best;
            }
        }
        best = wave_reduce<64>(best, MaxOp{});
        if (lane == 0)
            red[wave] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w)
            best = MaxOp{}(best, red[w]);
        if (threadIdx.x == 0)
            *out = uint2{(uint32_t)best, (uint32_t)(best >> 32)};
        return;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        row.values(raw[i], pos0 + i * kThreads * 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = fmaxf(m, x[e]);
    }
    // each wave by its own maximum, then the four
    m = wave_reduce<64>(m, MaxOp{});
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        row.values(raw[i], pos0 + i * kThreads * 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum += __builtin_amdgcn_exp2f((x[e] - base) * c);
    }
    sum = wave_reduce<64>(sum, SumOp{});
    float2 *mine = reinterpret_cast<float2 *>(red);
    if (lane == 0)
        mine[wave] = float2{m, sum};
    __syncthreads();
    if (threadIdx.x == 0) {
        float top = m;
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w)
            top = fmaxf(top, mine[w].x);
        const float all = top == -INFINITY ? 0.f : top;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w)
            sum += mine[w].y * __builtin_amdgcn_exp2f((mine[w].x - all) * c);
        *out = uint2{__builtin_bit_cast(uint32_t, top), __builtin_bit_cast(uint32_t, sum)};
    }
}

// A node's distribution as the walk keeps it: exp2((x - m) c) * inv.
struct Terms {
    float m, inv;
};

template <int DT>
__global__ __launch_bounds__(kWalkThreads) void tree_walk(KArgs a) {
    __shared__ float red[kWalkThreads / 64];
    __shared__ Terms p[kNodes], q[kNodes];
    __shared__ int32_t best[kNodes], token[kNodes], parent[kNodes], gone[kNodes];
    __shared__ float u[kNodes], px[kNodes], qx[kNodes];  // of a node's token, in its parent's rows
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x, lane = tid & 63, wave = wave_id();
    const int nodes = live_nodes(a, b);
    int32_t *tokens = a.tokens_out + (int64_t)b * a.n, *path = a.path_out + (int64_t)b * a.n;
    const float c = exponent_scale(a, b);
    if (tid < a.n) {
        tokens[tid] = -1;
        path[tid] = -1;
        token[tid] = a.node_tokens[(int64_t)b * a.n + tid];
        parent[tid] = tid > 0 && tid < nodes ? parent_of(a, b, tid) : -1;
        u[tid] = a.uniforms[(int64_t)b * a.n + tid];
    }
    // Join the chunks, sixteen lanes per row; the rows of leaves' drafters
    // hold nothing and are not looked at later.
    const int rows = a.draft && c != 0.f ? 2 * nodes : nodes;
    for (int r = tid / kJoinLanes; r < rows; r += kWalkThreads / kJoinLanes) {
        const int v = r < nodes ? r : r - nodes, sub = tid % kJoinLanes;
        const uint2 *part = a.part + (((int64_t)b * 2 + (r < nodes ? 0 : 1)) * a.n + v) * a.chunks;
        if (c == 0.f) {
            uint64_t k = 0;
            for (int x = sub; x < a.chunks; x += kJoinLanes)
                k = MaxOp{}(k, ((uint64_t)part[x].y << 32) | part[x].x);
            k = wave_reduce<kJoinLanes>(k, MaxOp{});
            if (sub == 0)
                best[v] = (int32_t)~(uint32_t)k;
            continue;
        }
        float m = -INFINITY, sum = 0.f;
        for (int x = sub; x < a.chunks; x += kJoinLanes) {
            const float mx = __builtin_bit_cast(float, part[x].x), lx = __builtin_bit_cast(float, part[x].y);
            const float top = fmaxf(m, mx), base = top == -INFINITY ? 0.f : top;
            sum = sum * __builtin_amdgcn_exp2f((m - base) * c) + lx * __builtin_amdgcn_exp2f((mx - base) * c);
            m = top;
        }
        const float top = wave_reduce<kJoinLanes>(m, MaxOp{}), base = top == -INFINITY ? 0.f : top;
        sum = wave_reduce<kJoinLanes>(sum * __builtin_amdgcn_exp2f((m - base) * c), SumOp{});
        if (sub == 0)
            (r < nodes ? p : q)[v] = Terms{top, 1.f / sum};
    }
    __syncthreads();
    // What each drafted token has in its parent's rows.
    if (tid < nodes) {
        const int v = parent[tid], x = token[tid];
        px[tid] = qx[tid] = 0.f;
        if (tid > 0 && v >= 0 && v < tid && c != 0.f && x >= 0 && x < a.vocab) {
            const int64_t at = ((int64_t)b * a.n + v) * a.vocab + x;
            px[tid] = __builtin_amdgcn_exp2f((logit_at<DT>(a.target, at) - p[v].m) * c) * p[v].inv;
            qx[tid] = a.draft ? __builtin_amdgcn_exp2f((logit_at<DT>(a.draft, at) - q[v].m) * c) * q[v].inv : 1.f;
        }
    }
    __syncthreads();
    int v = 0, count = 1, n_gone = 0;
    float S = 0.f;
    if (tid == 0 && nodes)
        path[0] = 0;
    for (bool more = nodes > 0; more;) {
        S = 0.f;
        n_gone = 0;
        float s = 1.f;
        bool stale = false;  // s is older than S
        int next = -1;
        for (int kid = v + 1; kid < nodes && next < 0; ++kid) {
            if (parent[kid] != v)
                continue;
            const int x = token[kid];
            if (c == 0.f) {
                next = x == best[v] ? kid : -1;
                continue;
            }
            if (stale) {
                const Row<DT> rp(a.target, a, b, v), rq(a.draft, a, b, v);
                float sum = 0.f;
                for (int pos = tid * 8; pos < rp.end(); pos += kPieces * kWalkThreads * 8) {
                    u32x4 wp[kPieces][Row<DT>::kElem / 2], wq[kPieces][Row<DT>::kElem / 2];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {  // past the row: zeros, left out as -inf
                        rp.load(pos + i * kWalkThreads * 8, wp[i]);
                        rq.load(pos + i * kWalkThreads * 8, wq[i]);
                    }
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        float xp[8], xq[8];
                        rp.values(wp[i], pos + i * kWalkThreads * 8, xp);
                        rq.values(wq[i], pos + i * kWalkThreads * 8, xq);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sum += left_of(__builtin_amdgcn_exp2f((xp[e] - p[v].m) * c) * p[v].inv, S,
                                           __builtin_amdgcn_exp2f((xq[e] - q[v].m) * c) * q[v].inv);
                    }
                }
                sum = wave_reduce<64>(sum, SumOp{});
                __syncthreads();
                if (lane == 0)
                    red[wave] = sum;
                __syncthreads();
                s = 0.f;
                for (int w = 0; w < kWalkThreads / 64; ++w)
                    s += red[w];
                stale = false;
            }
            float rx = a.draft ? left_of(px[kid], S, qx[kid]) : px[kid];
            for (int g = 0; g < n_gone; ++g)
                rx = gone[g] == x ? 0.f : rx;
            if (u[kid] * qx[kid] * s < rx) {
                next = kid;
            } else if (a.draft) {
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
        more = next >= 0;
        if (more) {
            if (tid == 0) {
                tokens[count - 1] = token[next];
                path[count] = next;
            }
            ++count;
            v = next;
        }
    }
    if (tid == 0) {
        a.count_out[b] = nodes ? count : 0;
        if (nodes && c == 0.f)
            tokens[count - 1] = best[v];
        Last &l = a.last[b];
        l.key = 0;
        l.arrived = 0;
        l.node = nodes && c != 0.f ? v : -1;
        l.at = count - 1;
        if (nodes) {
            l.m = p[v].m;
            l.inv = p[v].inv;
            l.mq = q[v].m;
            l.invq = q[v].inv;
        }
        l.S = S;
        l.n_gone = n_gone;
    }
    if (tid < n_gone)
        a.last[b].gone[tid] = gone[tid];
}

// The best key of a thread's tokens of one piece: argmax r / noise over r > 0.
// rest: the remainder (with S and the rejected tokens), else p itself.
template <int DT>
__device__ __forceinline__ uint64_t draw_piece(const KArgs &a, const Last &l, const Row<DT> &rp, const Row<DT> &rq,
                                               const float *noise, float c, int pos, bool rest) {
    const bool drawn = rest && l.S > 0.f;
    u32x4 wp[Row<DT>::kElem / 2], wq[Row<DT>::kElem / 2];
    float e8[8], xp[8], xq[8];
    rp.load(pos, wp);
    if (drawn)
        rq.load(pos, wq);
    const int x0 = pos - rp.shift;
    if (x0 >= 0 && x0 + 8 <= a.vocab) {
        typedef f32x4 f32x4_dword __attribute__((aligned(4)));  // the row may begin anywhere
        const f32x4 lo = *reinterpret_cast<const f32x4_dword *>(noise + x0),
                    hi = *reinterpret_cast<const f32x4_dword *>(noise + x0 + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            e8[e] = lo[e];
            e8[e + 4] = hi[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            e8[e] = x0 + e >= 0 && x0 + e < a.vocab ? noise[x0 + e] : 1.f;
    }
    rp.values(wp, pos, xp);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        xp[e] = __builtin_amdgcn_exp2f((xp[e] - l.m) * c) * l.inv;
    if (drawn) {
        rq.values(wq, pos, xq);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            xp[e] = left_of(xp[e], l.S, __builtin_amdgcn_exp2f((xq[e] - l.mq) * c) * l.invq);
    }
    if (rest)
        for (int g = 0; g < l.n_gone; ++g) {
            const int at = l.gone[g] - x0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                xp[e] = at == e ? 0.f : xp[e];
        }
    uint64_t best = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (xp[e] > 0.f) {
            const uint64_t k = key_of(xp[e] / e8[e], x0 + e);
            best = k > best ? k : best;
        }
    return best;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void tree_draw(KArgs a) {
    __shared__ uint64_t red[kThreads / 64];
    __shared__ int last_here;
    const int b = (int)blockIdx.y, tid = (int)threadIdx.x;
    Last &l = a.last[b];
    const int v = l.node;
    if (v < 0)
        return;
    const float c = exponent_scale(a, b);
    const Row<DT> rp(a.target, a, b, v), rq(a.draft ? a.draft : a.target, a, b, v);
    const float *noise = a.noise + (int64_t)b * a.vocab;
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pos = (int)blockIdx.x * kDrawChunk + (i * kThreads + tid) * 8;
        if (pos < rp.end())
            best = MaxOp{}(best, draw_piece<DT>(a, l, rp, rq, noise, c, pos, true));
    }
    best = wave_reduce<64>(best, MaxOp{});
    if ((tid & 63) == 0)
        red[tid >> 6] = best;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kThreads / 64; ++w)
            best = MaxOp{}(best, red[w]);
        // the key is in memory before this workgroup counts itself in: the
        // count waits for the value that the maximum replaced
        uint64_t old = __hip_atomic_fetch_max(&l.key, best, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" : "+v"(old)::"memory");
        last_here = __hip_atomic_fetch_add(&l.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                    gridDim.x - 1;
    }
    __syncthreads();
    if (!last_here)
        return;
    uint64_t key = __hip_atomic_load(&l.key, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (key == 0) {
        // nothing is left of r: p stands in
        for (int pos = tid * 8; pos < rp.end(); pos += kThreads * 8)
            key = MaxOp{}(key, draw_piece<DT>(a, l, rp, rq, noise, c, pos, false));
        key = wave_reduce<64>(key, MaxOp{});
        __syncthreads();
        if ((tid & 63) == 0)
            red[tid >> 6] = key;
        __syncthreads();
        for (int w = 0; w < kThreads / 64; ++w)
            key = MaxOp{}(key, red[w]);
    }
    if (tid == 0)
        a.tokens_out[(int64_t)b * a.n + l.at] = key ? (int32_t)~(uint32_t)key : 0;
}

// Chunks of a row: the first may begin with the 7 elements of alignment.
int row_chunks(int vocab) { return (vocab + 7 + kChunk - 1) / kChunk; }

template <int DT>
void launch_dt(const KArgs &a, int batch, hipStream_t stream) {
    hipLaunchKernelGGL(tree_row_stats<DT>, dim3(a.chunks, a.draft ? 2 * a.n : a.n, batch), dim3(kThreads), 0, stream,
                       a);
    hipLaunchKernelGGL(tree_walk<DT>, dim3(batch), dim3(kWalkThreads), 0, stream, a);
    hipLaunchKernelGGL(tree_draw<DT>, dim3((a.vocab + 7 + kDrawChunk - 1) / kDrawChunk, batch), dim3(kThreads), 0,
                       stream, a);
}

size_t part_bytes(int batch, int n, int vocab) {
    return ((size_t)batch * 2 * n * row_chunks(vocab) * sizeof(uint2) + 15) & ~(size_t)15;
}

}  // namespace

size_t tree_verify_workspace(int batch, int n, int vocab) {
    return part_bytes(batch, n, vocab) + (size_t)batch * sizeof(Last);
}

hipError_t launch_tree_verify(const TreeVerifyArgs &p) {
    KArgs a{p.target, p.draft, p.node_tokens, p.parents, p.n_nodes, p.temperature, p.uniforms, p.noise,
            p.tokens_out, p.path_out, p.count_out, static_cast<uint2 *>(p.workspace),
            reinterpret_cast<Last *>(static_cast<char *>(p.workspace) + part_bytes(p.batch, p.n, p.vocab)),
            p.n, p.vocab, row_chunks(p.vocab)};
    if (p.dtype == VQ_DTYPE_F32)
        launch_dt<VQ_DTYPE_F32>(a, p.batch, p.stream);
    else if (p.dtype == VQ_DTYPE_BF16)
        launch_dt<VQ_DTYPE_BF16>(a, p.batch, p.stream);
    else
        launch_dt<VQ_DTYPE_F16>(a, p.batch, p.stream);
    return hipGetLastError();
}

}  // namespace vq
