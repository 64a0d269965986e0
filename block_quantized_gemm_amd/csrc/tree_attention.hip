// tree_attention.hip -- attention of a tree of drafted tokens over a paged cache.
//
// For each query row (node i of sequence b, query head h):
//   out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  s_t = scale * (q . k_t),
// over the cached positions t < ctx_len[b] and the nodes its mask names, in
// one pass with a base m that follows the running maximum, and a sum l: when m
// grows, what was summed is multiplied by exp(m_old - m_new).
//
// The rows of one sequence that share a key/value head (nodes x query heads of
// the head's group) are the 16 columns of MFMA tiles, 32 tokens a step:
//   S^T [token][row] = K Q^T      two 16x16 tiles, D / 32 instructions each
//   O^T [channel][row] += V^T P^T D / 16 tiles, one instruction each
// Row r of the score tile a is token 8 (r / 4) + 4 a + r % 4 of the step, so
// that a lane (column j, group g) ends with the scores of tokens 8 g .. 8 g + 7
// of its row: exactly the eight k values it has to feed to the second product.
// The probabilities never leave the lane, and everything kept per row (m, l,
// the factor of O) is a lane's own register.  V^T comes from the cache as it
// lies there (transposed in blocks of 32 tokens), so no operand passes through
// LDS: each wave streams its own steps from memory into registers.
//
// Work is cut evenly whatever the sequences' lengths: the steps of all
// (sequence, head) pairs, laid end to end, are divided into equal ranges, one
// workgroup each (times the groups of query rows, whose workgroups sit next to
// each other on one XCD and read the same keys).  The four waves of a
// workgroup take its steps in turn and join through LDS; a pair cut by a range
// boundary leaves its pieces (m, l, O in fp32) in the workspace, and a second
// kernel joins them in order.
//
// Measured on one MI355X (whole call, bf16 unless noted; the rate is the cached
// keys and values, once, over that time), and each kernel's median in a trace,
// whose own overhead is in it:
//                                                              call            main    join
//   1 sequence, 8-node chain, 509 tokens, 64 / 8 heads of 128   23 us           18.4    4.5
//   32 sequences, single tokens, up to 4k, 32 / 8 of 64, f16    45 to 49        41.0    5.4   2.9 TB/s
//   8 sequences, 16-node trees, up to 16k, 64 / 8 of 128       144             142.1   10.8   2.3 TB/s
//   1 sequence, 16-node tree, 128k, 64 / 8 of 128              211             214.5    9.2   2.5 TB/s
//   4 sequences, 61-node trees, up to 8k, 32 / 4 of 256, f16   252 to 260      246.7    9.4
// What bounds them: with more rows than a workgroup holds (32, or 16 at D =
// 256) every group of rows reads the keys and values again.  L2 answers 1.25 GB
// of requests for the 8 trees and 2.18 GB for the 128k tree (four times the
// bytes; 9 and 10 TB/s) and sends 0.40 and 0.58 GB of them to memory; for the
// 61-node trees 2.0 to 2.4 GB (once per 16 rows; 8.5 TB/s) and 0.18 GB, and that
// kernel spills 51 registers.  The matrix units are busy 15% of the 128k call.
// Few rows: the page number of a step is read by a vector load and waited for,
// which also waits for the step's operands already on their way, so a wave has
// one step in flight.  The short chain is bound by the main kernel, not by its
// bytes (2.4 MB) nor by the host, since the two kernels fill the call: 68
// workgroups, each a chain of dependent steps (the scan, page numbers, operands,
// four-wave join), and the ranges that hold the end of one head and the start
// of the next go through two such chains.  Where in the chain the time goes has
// not been measured.
#include <atomic>

#include "tree_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;         // tokens per step
constexpr int kMinSteps = 4;      // steps per range at least: one per wave
// Probabilities are exp2(s - base).  The base is only raised when a score
// exceeds the row's maximum when it was set by more than this (in powers of
// two): until then the reduction over the row's four lanes and the scaling of O
// are skipped.
constexpr float kSlack = 8.f;
// The base lies this far below that maximum.  bf16 has fp32's exponents and
// needs none.  The probabilities that the second product takes in fp16 lose
// bits below 2^-14 and vanish below 2^-25, while their sum l, in fp32, keeps
// them: at base = maximum, 128k tokens that each hold 2^-25 of it drop 0.4% of
// the weight from O alone.  2^7 higher the largest is 2^(8 + 7), below fp16's
// 65504, and bits are lost only below 2^-21 of the maximum.
template <int DT>
constexpr float kLift = DT == VQ_DTYPE_F16 ? 7.f : 0.f;

struct KArgs {
    const uint16_t *q, *k, *v, *k_cache, *v_cache;
    const int32_t *page_table, *ctx_len;
    const uint64_t *tree_mask;
    const int32_t *n_nodes;
    uint16_t *out;
    float *pieces;       // [range * row groups + group][2] slots
    struct JoinDesc *join;
    int64_t q_stride, k_stride, v_stride;
    int batch, n, q_heads, kv_heads, page_shift, n_pages, max_pages;
    int ranges, row_groups;
    float scale_log2;    // scale * log2(e)
};

// A cut (sequence, head) pair and row group, as its first piece's workgroup
// leaves it for the joining kernel: the pieces are slot `first_slot` and the
// even slots of the next `count - 1` ranges.  count 0: nothing to join.
struct JoinDesc {
    int32_t b, h, first_slot, count;
};

template <int D, int QT>
struct Shape {
    static constexpr int kRows = 16 * QT;
    static constexpr int kSlotFloats = kRows * D + 2 * kRows;  // O in lane order, then m and l of each row
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kRowPitch = 2 * D + 16;  // a node's values in LDS, padded against bank conflicts
    static constexpr int kWaveBytes = kStep * kRowPitch;  // a wave's LDS: a step of node values, or 16 rows of O
    static constexpr int kJoinBytes = kWaves * (kWaveBytes + 16 * 4);
    static_assert(kWaveBytes >= 16 * D * 4, "a wave's part of O fits");
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = (uint32_t)uniform((int)(uint32_t)x), hi = (uint32_t)uniform((int)(uint32_t)((uint64_t)x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

template <int DT>
__device__ __forceinline__ float to_f32(uint32_t h) {
    if constexpr (DT == VQ_DTYPE_BF16)
        return __builtin_bit_cast(float, h << 16);
    else
        return h2f(h);
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if constexpr (DT == VQ_DTYPE_BF16) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(x), static_cast<__bf16>(y)});
    } else {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(x), static_cast<_Float16>(y)});
    }
}
// Whether a 16-bit value is infinite or NaN.
template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t h) {
    constexpr uint32_t kExp = DT == VQ_DTYPE_BF16 ? 0x7F80u : 0x7C00u;
    return (h & kExp) == kExp;
}

// Reductions over the four lanes that hold one row.
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16, 64));
    return fmaxf(x, __shfl_xor(x, 32, 64));
}
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

struct Sequence {
    int ctx, nodes, ctx_steps, steps;
};
__device__ __forceinline__ Sequence sequence(const KArgs &a, int b) {
    Sequence s;
    s.ctx = min(max(a.ctx_len[b], 0), a.max_pages << a.page_shift);
    s.nodes = a.n_nodes ? min(max(a.n_nodes[b], 0), a.n) : a.n;
    s.ctx_steps = (s.ctx + kStep - 1) / kStep;
    s.steps = s.nodes ? s.ctx_steps + (s.nodes + kStep - 1) / kStep : 0;
    return s;
}

// The nodes that row i of sequence b sees, as bits.
__device__ __forceinline__ uint64_t visible_nodes(const KArgs &a, int b, int i, int nodes) {
    if (i >= nodes)
        return 0;
    const uint64_t m = a.tree_mask ? a.tree_mask[(int64_t)b * a.n + i] : ~0ull >> (63 - i);
    return m & (~0ull >> (64 - nodes));
}

// Where the result of a row that summed to zero comes from: a row that sees
// nothing is zero; one whose every score is -inf is 0 / 0.
__device__ __forceinline__ float norm_of(float l, int ctx, uint64_t seen) {
    return l == 0.f && ctx == 0 && seen == 0 ? 0.f : 1.f / l;
}

// One wave's state over a (sequence, head) pair: D / 16 channel tiles of O^T
// for QT tiles of 16 rows, and each row's base (in powers of two, equal in its
// four lanes) and this lane's part of its sum.
template <int D, int QT>
struct Acc {
    f32x4 o[QT][D / 16];
    float m[QT], l[QT];
};

template <int DT, int D, int QT>
struct Wave {
    using A16 = Act16<DT>;
    static constexpr int kDs = D / 32, kDt = D / 16;

    u32x4 kf[2][kDs], vf[kDt];

    __device__ __forceinline__ void load_k(rsrc_t r, int row_bytes, int lane) {
        const int j = lane & 15, g = lane >> 4;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ds = 0; ds < kDs; ++ds)
                kf[t][ds] = bload16<kAuxCached>(r, (8 * (j >> 2) + 4 * t + (j & 3)) * row_bytes + 64 * ds + 16 * g, 0);
    }
    __device__ __forceinline__ void load_v(rsrc_t r, int lane) {
        const int at = (lane & 15) * (2 * kVBlock) + 16 * (lane >> 4);
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt)
            vf[dt] = bload16<kAuxCached>(r, at + (dt & 3) * (32 * kVBlock), (dt & ~3) * (32 * kVBlock));
    }
    // Values from rows (the nodes' own), by way of this wave's LDS: lane
    // (j, g) takes channel 16 dt + j of rows 8 g .. 8 g + 7.  Infinite and NaN
    // values are left out (zero); returns whether there were any.
    __device__ __forceinline__ bool load_v_rows(rsrc_t r, int row_bytes, uint8_t *lds, int lane) {
        constexpr int kPitch = Shape<D, 1>::kRowPitch, kRowLanes = D / 8, kRows = 64 / kRowLanes;
        bool wild = false;
        u32x4 f[kStep / kRows];
#pragma unroll
        for (int x = 0; x < kStep / kRows; ++x)
            f[x] = bload16<kAuxCached>(r, (x * kRows + lane / kRowLanes) * row_bytes + 16 * (lane % kRowLanes), 0);
#pragma unroll
        for (int x = 0; x < kStep / kRows; ++x) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t two = f[x][e];
                const bool lo = not_finite<DT>(two), hi = not_finite<DT>(two >> 16);
                f[x][e] = two & ((lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u));
                wild = wild || lo || hi;
            }
            *reinterpret_cast<u32x4 *>(lds + (x * kRows + lane / kRowLanes) * kPitch + 16 * (lane % kRowLanes)) = f[x];
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the other lanes' writes
        const uint8_t *at = lds + 8 * (lane >> 4) * kPitch + 2 * (lane & 15);
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                vf[dt][x] = (uint32_t) * reinterpret_cast<const uint16_t *>(at + 2 * x * kPitch + 32 * dt) |
                            (uint32_t) * reinterpret_cast<const uint16_t *>(at + (2 * x + 1) * kPitch + 32 * dt) << 16;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // before the next step's writes
        return __any(wild);
    }

    __device__ __forceinline__ void scores(const u32x4 *qlds, int qt, int lane, f32x4 (&s)[2]) const {
        s[0] = s[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ds = 0; ds < kDs; ++ds) {
            const u32x4 qf = qlds[(qt * kDs + ds) * 64 + lane];
            s[0] = A16::mfma(kf[0][ds], qf, s[0]);
            s[1] = A16::mfma(kf[1][ds], qf, s[1]);
        }
    }

    // Folds eight scores of each lane's row (already in powers of two, -inf
    // where unseen) into the base and sum; returns the probabilities in the
    // values' type, the operand type of the second product.
    __device__ __forceinline__ u32x4 fold(const float (&s)[8], int qt, Acc<D, QT> &acc) const {
        float top = s[0];
#pragma unroll
        for (int x = 1; x < 8; ++x)
            top = fmaxf(top, s[x]);
        constexpr float kRoom = kLift<DT> + kSlack;
        // by the difference, which is the probabilities' exponent to the bit: a
        // sum rounds where neighbouring floats are more than 1 apart
        if (__any(top - acc.m[qt] > kRoom)) {
            // row by row: a row keeps its base, and with it the rounding of
            // its probabilities, when only its neighbours exceed theirs
            const float most = row_max(top), m_new = most - acc.m[qt] > kRoom ? most - kLift<DT> : acc.m[qt];
            const float shrink = m_new == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(acc.m[qt] - m_new);
            acc.m[qt] = m_new;
            acc.l[qt] *= shrink;
#pragma unroll
            for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc.o[qt][dt][r] *= shrink;
        }
        const float base = acc.m[qt] == -INFINITY ? 0.f : acc.m[qt];
        float p[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
            p[x] = __builtin_amdgcn_exp2f(s[x] - base);
        acc.l[qt] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        return u32x4{pack2<DT>(p[0], p[1]), pack2<DT>(p[2], p[3]), pack2<DT>(p[4], p[5]), pack2<DT>(p[6], p[7])};
    }

    __device__ __forceinline__ void add_values(u32x4 p, int qt, Acc<D, QT> &acc) const {
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt)
            acc.o[qt][dt] = A16::mfma(vf[dt], p, acc.o[qt][dt]);
    }
};

// Processes steps [s0, s1) of pair (b, h) for row group rg: each wave takes
// every kWaves-th step.
template <int DT, int D, int QT>
__device__ __forceinline__ void run_steps(const KArgs &a, const Sequence &sq, int b, int h, int rg, int s0, int s1,
                                          const u32x4 *qlds, uint8_t *wave_lds, Acc<D, QT> &acc) {
    constexpr int kBlockBytes = kStep * D * 2;  // 32 tokens of one head: keys, and values, are contiguous in a page
    const int lane = (int)(threadIdx.x & 63), wave = wave_id(), j = lane & 15, g = lane >> 4;
    const int group = a.q_heads / a.kv_heads;
    Wave<DT, D, QT> w;
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        acc.m[qt] = -INFINITY;
        acc.l[qt] = 0.f;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
            acc.o[qt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t *table = a.page_table + (int64_t)b * a.max_pages;
    const int steps_shift = a.page_shift - 5;
    // Element offset of a step's block, the same in both caches; -1 for a page
    // outside the pool, which reads as zeros.
    auto block_at = [&](int s) -> int64_t {
        const int page = uniform(table[s >> steps_shift]);
        if (page < 0 || page >= a.n_pages)
            return -1;
        return ((((int64_t)page * a.kv_heads + h) << a.page_shift) + ((s & ((1 << steps_shift) - 1)) << 5)) * D;
    };
    auto rsrc_of = [&](const uint16_t *cache, int64_t at) {
        return make_rsrc(cache + (at < 0 ? 0 : at), at < 0 ? 0u : (uint32_t)kBlockBytes);
    };

    // Whole steps of the context: the next step's keys are on their way while
    // this one's probabilities are formed, its values while the next scores are.
    const int whole = min(s1, sq.ctx / kStep);
    int s = s0 + wave;
    if (s < whole) {
        int64_t at = block_at(s);
        w.load_k(rsrc_of(a.k_cache, at), D * 2, lane);
        w.load_v(rsrc_of(a.v_cache, at), lane);
        for (;;) {
            const int next = s + kWaves;
            const int64_t at_next = next < whole ? block_at(next) : -1;
            u32x4 p[QT];
            f32x4 sc[QT][2];
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
                w.scores(qlds, qt, lane, sc[qt]);
            __builtin_amdgcn_sched_barrier(0);
            w.load_k(rsrc_of(a.k_cache, at_next), D * 2, lane);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = sc[qt][e >> 2][e & 3] * a.scale_log2;
                p[qt] = w.fold(x, qt, acc);
            }
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
                w.add_values(p[qt], qt, acc);
            __builtin_amdgcn_sched_barrier(0);
            w.load_v(rsrc_of(a.v_cache, at_next), lane);
            __builtin_amdgcn_sched_barrier(0);
            s = next;
            if (s >= whole)
                break;
        }
    }

    // The context's last, partial step, and the nodes: positions are masked one
    // by one.  What nothing sees is taken out of the values too, because the
    // product would turn its infinities and NaN times zero into NaN.
    for (; s < s1; s += kWaves) {
        const bool tree = s >= sq.ctx_steps;
        const int first = tree ? (s - sq.ctx_steps) * kStep : s * kStep;
        const int count = (tree ? sq.nodes : sq.ctx) - first;  // positions of this step that exist
        bool wild = false;  // some value of a node is infinite or NaN
        rsrc_t rv;
        if (tree) {
            const int rows = min(count, kStep);
            const int64_t row = (int64_t)b * a.n + first;
            const rsrc_t rk = make_rsrc(a.k + row * a.k_stride + (int64_t)h * D,
                                        (uint32_t)(((int64_t)(rows - 1) * a.k_stride + D) * 2));
            rv = make_rsrc(a.v + row * a.v_stride + (int64_t)h * D,
                           (uint32_t)(((int64_t)(rows - 1) * a.v_stride + D) * 2));
            w.load_k(rk, (int)a.k_stride * 2, lane);
            wild = w.load_v_rows(rv, (int)a.v_stride * 2, wave_lds, lane);
        } else {
            const int64_t at = block_at(s);
            w.load_k(rsrc_of(a.k_cache, at), D * 2, lane);
            w.load_v(rsrc_of(a.v_cache, at), lane);
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    w.vf[dt][x] &= (8 * g + 2 * x < count ? 0xFFFFu : 0u) |
                                   (8 * g + 2 * x + 1 < count ? 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            f32x4 sc[2];
            w.scores(qlds, qt, lane, sc);
            uint32_t seen;  // bit x: the row sees position first + 8 g + x
            if (tree) {
                const int i = (rg * Shape<D, QT>::kRows + 16 * qt + j) / group;
                seen = (uint32_t)(visible_nodes(a, b, i, sq.nodes) >> (first + 8 * g));
            } else {
                seen = count >= 8 * g + 8 ? 0xFFu : count <= 8 * g ? 0u : 0xFFu >> (8 * g + 8 - count);
            }
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = (seen >> e & 1) ? sc[e >> 2][e & 3] * a.scale_log2 : -INFINITY;
            w.add_values(w.fold(x, qt, acc), qt, acc);
            if (wild) {
                // the infinite and NaN values, element by element, for the rows that see them
                const float base = acc.m[qt] == -INFINITY ? 0.f : acc.m[qt];
                for (int t = 0; t < kStep; ++t) {
                    const int src = (lane & 15) | ((t >> 3) << 4);
                    float pt = 0.f;
                    bool sees = false;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if ((t & 7) == e) {
                            pt = __shfl(__builtin_amdgcn_exp2f(x[e] - base), src, 64);
                            sees = __shfl((int)(seen >> e & 1), src, 64) != 0;
                        }
#pragma unroll
                    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t hv =
                                bload2<kAuxCached>(rv, t * (int)a.v_stride * 2 + 2 * (16 * dt + 4 * g + r), 0);
                            if (sees && not_finite<DT>(hv))
                                acc.o[qt][dt][r] += pt * to_f32<DT>(hv);
                        }
                }
            }
        }
    }
#pragma unroll
    for (int qt = 0; qt < QT; ++qt)
        acc.l[qt] = row_sum(acc.l[qt]);
}

// Joins the waves' states in wave order and writes the rows out, or, for a
// part of the pair's steps, the joined piece.
template <int DT, int D, int QT>
__device__ __forceinline__ void join_waves(const KArgs &a, const Sequence &sq, int b, int h, int rg, bool whole,
                                           float *slot, uint8_t *lds, Acc<D, QT> &acc) {
    constexpr int kDt = D / 16, kRows = Shape<D, QT>::kRows;
    const int lane = (int)(threadIdx.x & 63), wave = wave_id(), j = lane & 15, g = lane >> 4;
    const int group = a.q_heads / a.kv_heads;
    f32x4 *ol = reinterpret_cast<f32x4 *>(lds);                       // [wave][dt][lane]
    float *ml = reinterpret_cast<float *>(lds + kWaves * Shape<D, QT>::kWaveBytes);  // [wave][row]
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        __syncthreads();
        if (g == 0)
            ml[wave * 16 + j] = acc.m[qt];
        __syncthreads();
        float m = ml[j];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            m = fmaxf(m, ml[w * 16 + j]);
        const float shrink = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(acc.m[qt] - m);
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt)
            ol[(wave * kDt + dt) * 64 + lane] = acc.o[qt][dt] * shrink;
        __syncthreads();
        if (g == 0)
            ml[wave * 16 + j] = acc.l[qt] * shrink;
        __syncthreads();
        float l = ml[j];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
            l += ml[w * 16 + j];
        const int row = rg * kRows + 16 * qt + j, i = row / group;
        const float inv = whole ? norm_of(l, sq.ctx, visible_nodes(a, b, i, sq.nodes)) : 1.f;
        for (int dt = wave; dt < kDt; dt += kWaves) {
            f32x4 o = ol[dt * 64 + lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                o += ol[(w * kDt + dt) * 64 + lane];
            if (!whole) {
                reinterpret_cast<f32x4 *>(slot)[(qt * kDt + dt) * 64 + lane] = o;
            } else if (row < sq.nodes * group) {
                uint16_t *dst = a.out + (((int64_t)b * a.n + i) * a.q_heads + h * group + (row - i * group)) * D +
                                16 * dt + 4 * g;
                *reinterpret_cast<u32x2 *>(dst) =
                    u32x2{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
            }
        }
        if (!whole && wave == 0 && g == 0) {
            slot[kRows * D + 16 * qt + j] = m;
            slot[kRows * D + kRows + 16 * qt + j] = l;
        }
    }
}

template <int DT, int D, int QT>
__global__ __launch_bounds__(kThreads, 2) void tree_attention_kernel(KArgs a) {
    using S = Shape<D, QT>;
    __shared__ __align__(16) uint8_t lds[S::kQBytes + S::kJoinBytes];
    __shared__ int64_t scan[kThreads];
    __shared__ int64_t found_at;
    __shared__ int found_b;
    const int tid = (int)threadIdx.x, wave = wave_id(), lane = tid & 63;
    const int group = a.q_heads / a.kv_heads;
    const int run = xcd_run_index((int)blockIdx.x, (int)gridDim.x);
    const int range = run / a.row_groups, rg = run - range * a.row_groups;
    if (tid == 0)
        a.join[run].count = 0;

    // Rows past a sequence's nodes are zero.
    if (a.n_nodes)
        for (int b = (int)blockIdx.x; b < a.batch; b += (int)gridDim.x) {
            const int nodes = min(max(a.n_nodes[b], 0), a.n);
            u32x4 *p = reinterpret_cast<u32x4 *>(a.out + ((int64_t)b * a.n + nodes) * a.q_heads * D);
            const int pieces = (a.n - nodes) * a.q_heads * (D / 8);
            for (int x = tid; x < pieces; x += kThreads)
                p[x] = u32x4{0u, 0u, 0u, 0u};
        }

    // This workgroup's range of steps: all sequences' steps added up, each
    // thread a run of consecutive sequences.
    const int per = (a.batch + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int x = 0; x < per; ++x)
        if (tid * per + x < a.batch)
            mine += (int64_t)sequence(a, tid * per + x).steps * a.kv_heads;
    scan[tid] = mine;
    __syncthreads();
    for (int off = 1; off < kThreads; off <<= 1) {
        const int64_t add = tid >= off ? scan[tid - off] : 0;
        __syncthreads();
        scan[tid] += add;
        __syncthreads();
    }
    const int64_t total = uniform(scan[kThreads - 1]);
    const int64_t share = total <= (int64_t)a.ranges * kMinSteps ? kMinSteps : (total + a.ranges - 1) / a.ranges;
    int64_t u = range * share;
    const int64_t u_end = min(total, u + share);
    if (u >= u_end)
        return;
    if (scan[tid] > u && scan[tid] - mine <= u) {
        int64_t at = scan[tid] - mine;
        for (int x = 0; x < per; ++x) {
            const int64_t units = (int64_t)sequence(a, tid * per + x).steps * a.kv_heads;
            if (at + units > u) {
                found_b = tid * per + x;
                found_at = at;
                break;
            }
            at += units;
        }
    }
    __syncthreads();
    int b = uniform(found_b);
    int64_t off = u - uniform(found_at);
    const u32x4 *qlds = reinterpret_cast<const u32x4 *>(lds);
    bool first = true;

    while (u < u_end) {
        const Sequence sq = sequence(a, b);
        if (off >= (int64_t)sq.steps * a.kv_heads) {
            off -= (int64_t)sq.steps * a.kv_heads;
            ++b;
            continue;
        }
        const int h = (int)(off / sq.steps), s0 = (int)(off - (int64_t)h * sq.steps);
        const int s1 = (int)min((int64_t)sq.steps, s0 + (u_end - u));
        if (rg * S::kRows < sq.nodes * group) {
            // the rows' queries in the order the lanes feed them: [qt][ds][lane]
            for (int x = wave; x < QT * (D / 32); x += kWaves) {
                const int qt = x / (D / 32), ds = x % (D / 32);
                const int row = rg * S::kRows + 16 * qt + (lane & 15), i = row / group;
                u32x4 f = u32x4{0u, 0u, 0u, 0u};
                if (row < sq.nodes * group)
                    f = ld16(a.q + ((int64_t)b * a.n + i) * a.q_stride + (int64_t)(h * group + row - i * group) * D +
                             32 * ds + 8 * (lane >> 4));
                reinterpret_cast<u32x4 *>(lds)[x * 64 + lane] = f;
            }
            __syncthreads();
            Acc<D, QT> acc;
            run_steps<DT, D, QT>(a, sq, b, h, rg, s0, s1, qlds, lds + S::kQBytes + wave * S::kWaveBytes, acc);
            const bool whole = s0 == 0 && s1 == sq.steps;
            const int slot = 2 * run + (first ? 0 : 1);
            join_waves<DT, D, QT>(a, sq, b, h, rg, whole, a.pieces + (int64_t)slot * S::kSlotFloats,
                                  lds + S::kQBytes, acc);
            if (s0 == 0 && !whole && tid == 0)
                a.join[run] = JoinDesc{b, h, slot,
                                       (int)(1 + (u + sq.steps - 1) / share - u / share)};
            __syncthreads();  // the queries' area is free for the next pair
        }
        u += s1 - s0;
        off += s1 - s0;
        first = false;
    }
}

// Joins the pieces of a cut pair, in order: one workgroup per (first piece's
// workgroup, row tile, channel tile), each wave a run of the pieces.
template <int DT, int D, int QT>
__global__ __launch_bounds__(kThreads) void tree_join_kernel(KArgs a) {
    using S = Shape<D, QT>;
    constexpr int kDt = D / 16;
    __shared__ f32x4 ol[kWaves][64];
    __shared__ float ml[kWaves][64], ll[kWaves][64];
    const int run = (int)blockIdx.x, tile = (int)blockIdx.y, qt = tile / kDt, dt = tile % kDt;
    const JoinDesc d = a.join[run];
    if (d.count == 0)
        return;
    const int lane = (int)(threadIdx.x & 63), wave = wave_id(), j = lane & 15, g = lane >> 4;
    const int range = run / a.row_groups, rg = run - range * a.row_groups, group = a.q_heads / a.kv_heads;
    const int per = (d.count + kWaves - 1) / kWaves, p0 = wave * per, p1 = min(d.count, p0 + per);
    auto slot_of = [&](int p) {
        return a.pieces + (int64_t)(p == 0 ? d.first_slot : 2 * ((range + p) * a.row_groups + rg)) * S::kSlotFloats;
    };
    float m = -INFINITY, l = 0.f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int kBatch = 8;  // pieces in flight
    for (int p = p0; p < p1; p += kBatch) {
        f32x4 op[kBatch];
        float mp[kBatch], lp[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const float *s = slot_of(min(p + x, p1 - 1));
            op[x] = reinterpret_cast<const f32x4 *>(s)[tile * 64 + lane];
            mp[x] = s[S::kRows * D + 16 * qt + j];
            lp[x] = s[S::kRows * D + S::kRows + 16 * qt + j];
        }
        float top = m;
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
            top = fmaxf(top, mp[x]);
        const float base = top == -INFINITY ? 0.f : top, shrink = __builtin_amdgcn_exp2f(m - base);
        m = top;
        l *= shrink;
        o *= shrink;
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
            if (p + x < p1) {
                const float f = __builtin_amdgcn_exp2f(mp[x] - base);
                l += lp[x] * f;
                o += op[x] * f;
            }
    }
    ol[wave][lane] = o;
    ml[wave][lane] = m;
    ll[wave][lane] = l;
    __syncthreads();
    if (wave != 0)
        return;
    float top = m;
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        top = fmaxf(top, ml[w][lane]);
    const float base = top == -INFINITY ? 0.f : top;
    l = 0.f;
    o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w][lane] - base);
        l += ll[w][lane] * f;
        o += ol[w][lane] * f;
    }
    const Sequence sq = sequence(a, d.b);
    const int row = rg * S::kRows + 16 * qt + j, i = row / group;
    if (row >= sq.nodes * group)
        return;
    const float inv = norm_of(l, sq.ctx, visible_nodes(a, d.b, i, sq.nodes));
    uint16_t *dst = a.out + (((int64_t)d.b * a.n + i) * a.q_heads + d.h * group + (row - i * group)) * D + 16 * dt +
                    4 * g;
    *reinterpret_cast<u32x2 *>(dst) = u32x2{pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv)};
}

constexpr int kMaxWorkgroups = 1024;

// Tiles of 16 query rows per wave, all four waves of a workgroup holding the
// same rows: as many as the rows need, up to what a wave's 256 registers hold
// beside a step of keys and values (two tiles of D = 128: 64 for O, 64 for the
// operands, 32 for the scores and probabilities; D = 256 needs 64 and 128 for
// one, and spills 51 as it is).  More rows per workgroup, and so less
// re-reading, would take waves with different rows.
int row_tiles(int rows, int D) {
    const int most = D == 256 ? 1 : 2;
    return rows <= 16 ? 1 : most;
}

int device_cus() {
    static std::atomic<int> cus{0};
    int c = cus.load(std::memory_order_relaxed);
    if (!c) {
        int dev = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || c < 1)
            c = 256;
        cus.store(c, std::memory_order_relaxed);
    }
    return c;
}

struct Plan {
    int tiles, row_groups, ranges;
};
// `groups` workgroups at most, a whole number of ranges.
Plan plan_of(int n, int q_heads, int kv_heads, int D, int groups) {
    Plan p;
    const int rows = n * (q_heads / kv_heads);
    p.tiles = row_tiles(rows, D);
    p.row_groups = (rows + 16 * p.tiles - 1) / (16 * p.tiles);
    p.ranges = std::max(1, groups / p.row_groups);
    return p;
}
size_t slot_bytes(int tiles, int D) { return (size_t)(16 * tiles * D + 32 * tiles) * 4; }
size_t join_bytes(const Plan &p) { return (size_t)p.ranges * p.row_groups * sizeof(JoinDesc); }

template <int DT, int D, int QT>
void launch_shape(const KArgs &a, hipStream_t stream) {
    const int grid = a.ranges * a.row_groups;
    hipLaunchKernelGGL((tree_attention_kernel<DT, D, QT>), dim3(grid), dim3(kThreads), 0, stream, a);
    hipLaunchKernelGGL((tree_join_kernel<DT, D, QT>), dim3(grid, QT * D / 16), dim3(kThreads), 0, stream, a);
}
template <int DT>
void launch_type(const KArgs &a, int D, int tiles, hipStream_t stream) {
    if (D == 64)
        tiles == 1 ? launch_shape<DT, 64, 1>(a, stream) : launch_shape<DT, 64, 2>(a, stream);
    else if (D == 128)
        tiles == 1 ? launch_shape<DT, 128, 1>(a, stream) : launch_shape<DT, 128, 2>(a, stream);
    else
        launch_shape<DT, 256, 1>(a, stream);
}

}  // namespace

size_t tree_attention_workspace(int batch, int n, int q_heads, int kv_heads, int head_dim) {
    (void)batch;
    const Plan p = plan_of(n, q_heads, kv_heads, head_dim, kMaxWorkgroups);
    return join_bytes(p) + (size_t)p.ranges * p.row_groups * 2 * slot_bytes(p.tiles, head_dim);
}

hipError_t launch_tree_attention(const TreeAttnArgs &p) {
    const Plan pl = plan_of(p.n, p.q_heads, p.kv_heads, p.head_dim, std::min(kMaxWorkgroups, 2 * device_cus()));
    KArgs a{};
    a.q = static_cast<const uint16_t *>(p.q);
    a.k = static_cast<const uint16_t *>(p.k);
    a.v = static_cast<const uint16_t *>(p.v);
    a.k_cache = static_cast<const uint16_t *>(p.k_cache);
    a.v_cache = static_cast<const uint16_t *>(p.v_cache);
    a.page_table = p.page_table;
    a.ctx_len = p.ctx_len;
    a.tree_mask = p.tree_mask;
    a.n_nodes = p.n_nodes;
    a.out = static_cast<uint16_t *>(p.out);
    a.join = static_cast<JoinDesc *>(p.workspace);
    a.pieces = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + join_bytes(pl));
    a.q_stride = p.q_stride;
    a.k_stride = p.k_stride;
    a.v_stride = p.v_stride;
    a.batch = p.batch;
    a.n = p.n;
    a.q_heads = p.q_heads;
    a.kv_heads = p.kv_heads;
    a.page_shift = __builtin_ctz((unsigned)p.page_size);
    a.n_pages = p.n_pages;
    a.max_pages = p.max_pages;
    a.ranges = pl.ranges;
    a.row_groups = pl.row_groups;
    a.scale_log2 = p.scale * 1.44269504088896f;
    if (p.dtype == VQ_DTYPE_BF16)
        launch_type<VQ_DTYPE_BF16>(a, p.head_dim, pl.tiles, p.stream);
    else
        launch_type<VQ_DTYPE_F16>(a, p.head_dim, pl.tiles, p.stream);
    return hipGetLastError();
}

}  // namespace vq
