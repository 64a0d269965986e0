// w8a8_gemm.hip -- int8 weights with a scale per output channel times int8
// activations with a scale per row, and the gated product of two of them.
//
//   dot[n][m] = sum_k x[n][k] w[m][k]   (32-bit integer, exact: K <= 131056)
//   out[n][m] = dot * sx[n] * sw[m] + bias[m]
//   gated:      act(dot_gate * sx * sg) * (dot_up * sx * su)
//
// The dot is an exact integer whatever the order of its terms, so every form
// below returns the same bits for a row, whatever the other rows, their
// number and the split of K.
//
// A workgroup computes BM rows x BF features with the 16x16x64 int8 MFMA,
// weights as the first operand: a lane then holds runs of consecutive features
// of one row, and in the gated form gate and up of the same feature.  Chunks
// of 128 k go straight into LDS, up to STAGES of them in flight or in use; the
// operands of a step are read while the one before it is multiplied.
//
// Persistent workgroups, one or two a CU: whole rounds of tiles first, then the
// tiles that are left, each cut along k into as many equal pieces as there are
// workgroups for (the last piece to arrive adds the others).  Equal pieces keep
// the workgroups of an XCD at the same k of neighbouring tiles, whose operands
// then meet in L2: even ranges over all chunks balance better on paper and
// took 313 us where whole tiles on 240 of 256 CUs took 210.
//
// Nine forms, chosen by their estimated time (kForms).  For few rows, groups of
// waves split a tile's k and each streams for itself, without barriers: 1 row
// 8192 to 5120 in 9.1 to 9.7 us (4.3 to 4.6 TB/s), 16 rows 5120 to 17408 in 19.3 to
// 20.9 us (4.3 to 4.7 TB/s, a copy reaches 4.9), gated 16 rows 17408 in 40 us, 61
// rows in 38; bound by the weights' bytes and 5 us of launch, first loads and last
// stores.  For many, 256 x 256 tiles: 4,093 rows 17408 to 5120 in 294 to 302 us
// (2,416 to 2,480 TOPS; the library int8 product of 8192^3 2,458), 4,096 rows to
// 8192 in 432 to 461, gated 2,048 rows in 316 to 322.  There the matrix
// instructions run 60% (4,093 rows) and 70% (4,096) of the time.  With parts left
// out, before the loads were spread between them, the loop of the 4,096 rows took
// 328 of then 437 us without the loads, 392 with loads that all hit L2, 293
// without LDS reads either.  Between the two, 64 to 1,000 rows take 1.4 to 2.3
// times their floor: tiles of 128 and 256 rows pad, and 128 x 128 ones bring a
// third more bytes into LDS than 256 x 128 (300 rows 17408 to 5120 44 us, floor
// 21.8).
#include <atomic>

#include "layer_internal.h"
#include "vq_device.h"
#include "w8a8_plan.h"

namespace vq {

namespace {

constexpr int kOutOfRange = 1 << 30;  // past every range below (and no sum with it overflows): the load returns zeros
constexpr int kCoherent = 0x10;          // sc1: agent-coherent, no cache maintenance needed
constexpr int kStrip = 4;                // feature columns of tiles walked together

struct KArgs {
    const int8_t *w, *up, *x;
    const float *w_scales, *up_scales, *x_scales, *bias;
    void *out;
    uint32_t *counters;  // and the pieces behind them
    int N, M, K, out_dtype, activation;
    int row_tiles, col_tiles;
    int whole;  // tiles that are computed whole, by the workgroups in turn
    int cuts;   // each of the others is cut along k into so many pieces
};

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0,
                                                 0);
}

// The activations are written so that no large term is subtracted from
// another: 0.5 g (1 + tanh z) = g / (1 + exp(-2 z)), and the Gaussian's
// distribution function as 0.5 erfc(-g / sqrt 2).  exp and the quotient are the
// hardware's base-2 power and reciprocal, one unit each.  The power's exponent t
// is fp32: its roundings, two for SiLU and five for the tanh form, are |t| ln 2
// times as large relative to the result.  For 16-bit outputs that is below 2^-15
// (|t| <= 126, beyond which the result is 0), a sixteenth of what their own
// rounding may move it; for fp32 outputs the tanh form has no fewer in the plain
// order of its formula, but SiLU has: there (FINE) the power is corrected by what
// the exponent's roundings took, which leaves it within 8 half units instead of
// 28 (g down to -31): 2,048 rows gated to fp32 347 us, 336 without.
__device__ __forceinline__ float over_one_plus_exp2(float g, float t) {  // g / (1 + 2^t)
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}
template <int KIND, bool FINE>
__device__ __forceinline__ float activate(float g) {
    constexpr float kLog2e = 1.4426950408889634f;
    if constexpr (KIND == VQ_ACT_SILU && FINE) {
        // |x| log2 e < 128: the power stays finite, and where it passes 2^126 its
        // reciprocal is 0
        constexpr float kMost = 88.72f, kLn2 = 0.6931471805599453f;
        constexpr float kLow = (float)(1.4426950408889634 - (double)kLog2e);
        const float x = __builtin_amdgcn_fmed3f(g, -kMost, kMost), t = -kLog2e * x;
        const float lost = __builtin_fmaf(-kLow, x, __builtin_fmaf(-kLog2e, x, -t));
        const float e = __builtin_amdgcn_exp2f(t);
        return g * __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, lost * kLn2, e));
    } else if constexpr (KIND == VQ_ACT_SILU) {
        return over_one_plus_exp2(g, -kLog2e * g);
    } else if constexpr (KIND == VQ_ACT_GELU_TANH) {
        constexpr float kA = -2.0f * kLog2e * 0.7978845608028654f, kB = kA * 0.044715f;
        return over_one_plus_exp2(g, g * __builtin_fmaf(kB * g, g, kA));
    } else {
        return 0.5f * g * erfcf(g * -0.7071067811865476f);
    }
}

// A wave's 16-byte LDS read takes four cycles of 16 lanes, the first two {0-3,
// 12-15, 20-27} and {4-11, 16-19, 28-31}, the others 32 lanes on (seen in the
// conflict counter).  Lane 16 g + j reads the 16 bytes 4 step + g of a row; two
// rows are 256 bytes, all 64 banks.  The slots of a row are XORed with a number
// that makes every cycle cover all banks once.
//
// Activations: lane j reads row j.
__device__ __forceinline__ int swizzle_x(int row) { return row >> 1 & 7; }
// Weights: which row of its wave's is feature j of tile ft.  In a pair of tiles
// lane group g gets features 8 g .. 8 g + 7, so that a row of outputs leaves in
// 16-byte pieces, 64 bytes side by side (4 and 32 made 134 MB of outputs take
// 111 us).
template <int FO>
__device__ __forceinline__ int row_w(int ft, int j) {
    return FO == 1 ? j : 32 * (ft >> 1) + 8 * (j >> 2) + 4 * (ft & 1) + (j & 3);
}
template <int FO>
__device__ __forceinline__ int swizzle_w(int row) {
    return FO == 1 ? row >> 1 & 7 : (row >> 3 & 3) << 1 | (row >> 1 & 1);
}

// A piece of work: chunks [c0, c1) of one tile.
struct Part {
    int tile, c0, c1;
};

// RT x FT tiles of 16 rows x 16 features per wave, WR x WF waves that share
// their operands, and WK such groups that share a tile's k: a chunk is WK
// times KC = 128 k, group i's the i-th 128, in STAGES stages.
// FINE: gated to fp32 (kernels of their own: one more epilogue beside the others
// slowed those, 2,048 rows to 16 bits from 319 to 327 us).
// AUX: the cache policy of the weights' loads.
template <int RT, int FT, int WR, int WF, int WK, int STAGES, bool GATED, bool FINE, int AUX>
__global__ __launch_bounds__(64 * WR * WF * WK) void w8a8_kernel(KArgs a) {
    constexpr int kWaves = WR * WF, BM = 16 * RT * WR, BF = 16 * FT * WF;
    constexpr int kWPieces = BF / 8, kXPieces = BM / 8;  // 1 KiB each, a wave's load: 8 rows of KC bytes
    constexpr int kPieces = kWPieces + kXPieces;
    constexpr int kPer = kPieces / kWaves, kExtra = kPieces % kWaves, kMost = kPer + (kExtra ? 1 : 0);
    constexpr int kStage = kPieces * 1024;  // of one group; each has its stages to itself
    constexpr int kOutFeats = GATED ? BF / 2 : BF;  // output features of the workgroup
    constexpr int FO = GATED ? FT / 2 : FT;         // output feature tiles of a wave
    constexpr int kSlot = BM * BF * 4;              // bytes of a tile's sums
    constexpr int kSteps = KC / 64;                 // MFMA steps of a chunk
    static_assert(WK * kWaves <= 8 && (kWaves == 1 || kWaves % 2 == 0) && (!GATED || FT % 2 == 0), "shape");
    static_assert(kWPieces % (GATED ? 2 * kWaves : kWaves) == 0, "a wave's i-th piece is of the same matrix in every wave");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
    const int wk = WK > 1 ? wave_id() / kWaves : 0, wave = WK > 1 ? wave_id() % kWaves : wave_id();
    const int wr = wave % WR, wf = wave / WR;
    const int G = (int)gridDim.x, me = xcd_run_index((int)blockIdx.x, G);
    const int K = a.K, nch = (K + WK * KC - 1) / (WK * KC);
    const int alone = a.whole / G + (me < a.whole % G ? 1 : 0);
    // the tiles after the whole ones, cut: the workgroups of one XCD, whose
    // numbers follow each other, work at the same k of neighbouring tiles
    const int rest = a.row_tiles * a.col_tiles - a.whole;
    const int parts = alone + (me < rest * a.cuts ? 1 : 0);
    if (parts == 0)
        return;
    const auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };  // kept in a scalar register
    const int my_cut = parts > alone ? uniform(me / rest) : 0;
    const int my_c0 = parts > alone ? uniform(my_cut * nch / a.cuts) : 0;
    const int my_c1 = parts > alone ? uniform((my_cut + 1) * nch / a.cuts) : 0;
    const auto part = [&](int i) -> Part {
        if (i < alone)
            return Part{i * G + me, 0, nch};
        return Part{a.whole + me - my_cut * rest, my_c0, my_c1};
    };
    // tiles in strips of kStrip feature columns, rows of a strip one after the
    // other: neighbours, which run on one XCD, share rows and columns in its L2
    const auto place = [&](int tile, int &fb, int &rb) {
        const int per = kStrip * a.row_tiles, strip = tile / per, in = tile - strip * per;
        const int width = min(kStrip, a.col_tiles - strip * kStrip);
        rb = in / width * BM;
        fb = (strip * kStrip + in % width) * kOutFeats;
    };

    // Piece p = wave + kWaves i of a group's chunk holds rows 8 p .. 8 p + 7 of
    // it; a row's 16-byte slot s holds its bytes 16 (s ^ swizzle(row)) .. +16.
    // The swizzles repeat every 32 rows (16 for the activations), with i.
    constexpr int kWKinds = kWaves >= 4 ? 1 : 4 / kWaves, kXKinds = kWaves >= 2 ? 1 : 2;
    const int prow = lane / 8;
    int wvoff[kWKinds], xvoff[kXKinds], xbyte[kXKinds];
#pragma unroll
    for (int o = 0; o < kWKinds; ++o)
        wvoff[o] = prow * K + 16 * ((lane & 7) ^ swizzle_w<FO>(8 * (wave + kWaves * o) + prow));
#pragma unroll
    for (int o = 0; o < kXKinds; ++o) {
        xbyte[o] = 16 * ((lane & 7) ^ swizzle_x(8 * (wave + kWaves * o) + prow));
        xvoff[o] = prow * K + xbyte[o];
    }
    rsrc_t rx, rw, ru;
    int at = -1, lc = 0, lend = 0;  // the part whose chunks are being loaded
    const auto open = [&]() {
        if (++at >= parts) {
            lc = -1;  // nothing left: what follows loads zeros
            return;
        }
        const Part p = part(at);
        int fb, rb;
        place(p.tile, fb, rb);
        lc = p.c0;
        lend = p.c1;
        const uint32_t feats = (uint32_t)min(kOutFeats, a.M - fb);
        rx = make_rsrc(a.x + (size_t)rb * K, (uint32_t)min(BM, a.N - rb) * (uint32_t)K);
        rw = make_rsrc(a.w + (size_t)fb * K, feats * (uint32_t)K);
        if constexpr (GATED)
            ru = make_rsrc(a.up + (size_t)fb * K, feats * (uint32_t)K);
    };
    uint8_t *mem = lds + wk * STAGES * kStage;
    // Loads of the chunk that comes next, kMost pieces of 1 KiB a wave: [I0, I1)
    // of them.
    const auto load = [&](int stage, auto I0, auto I1) {
        const int k0 = (max(lc, 0) * WK + wk) * KC;
        // past K the row's neighbour would be read: the activations are
        // zeros there, and so is the product
        const bool none = lc < 0 || k0 >= K;
        uint8_t *st = mem + stage * kStage + wave * 1024;
        const int step = kWaves * 8 * K;  // a wave's next piece
        const int base = wave * 8 * K + k0;
        static_for<I1.value - I0.value>([&](auto I) {
            constexpr int i = I0.value + I.value, x0 = kWPieces / kWaves, up0 = x0 / 2;
            if constexpr (i >= x0) {
                constexpr int o = (i - x0) % kXKinds;
                if (kExtra == 0 || i < kMost - 1 || wave < kExtra)
                    bload16_lds(rx, st + 1024 * kWaves * i, !none && k0 + xbyte[o] < K ? xvoff[o] : kOutOfRange,
                                base + (i - x0) * step);
            } else if constexpr (GATED && i >= up0) {
                bload16_lds<AUX>(ru, st + 1024 * kWaves * i, none ? kOutOfRange : wvoff[(i - up0) % kWKinds],
                            base + (i - up0) * step);
            } else {
                bload16_lds<AUX>(rw, st + 1024 * kWaves * i, none ? kOutOfRange : wvoff[i % kWKinds], base + i * step);
            }
        });
    };
    const auto loaded = [&]() {  // on to the next chunk
        if (lc >= 0 && ++lc == lend)
            open();
    };

    i32x4 acc[FT][RT];
    u32x4 xb[RT], wa[FT];
    const uint8_t *xs = mem + kWPieces * 1024 + (wr * RT * 16 + j) * KC, *ws = mem + wf * FO * 16 * KC;
    const auto read_x = [&](int s, int rt, int stage) {
        return *reinterpret_cast<const u32x4 *>(xs + stage * kStage + rt * 16 * KC + 16 * ((4 * s + g) ^ swizzle_x(j)));
    };
    const auto read_w = [&](int s, int ft, int stage) {
        const int row = row_w<FO>(ft % FO, j);
        return *reinterpret_cast<const u32x4 *>(ws + stage * kStage + ((ft < FO ? 0 : BF / 2) + row) * KC +
                                                16 * ((4 * s + g) ^ swizzle_w<FO>(row)));
    };
    // All but the newest C chunks' loads have landed, and every wave that reads
    // them holds what it read before.  A group of one wave waits for itself.
    int settled = 0;  // so many more chunks are known to have landed
    const auto landed = [&](auto C) {
        if (settled > 0)
            --settled;
        else if (!kExtra || wave >= kExtra)
            wait_vmcnt<C.value * kPer>();
        else
            wait_vmcnt<C.value * kMost>();
        if constexpr (kWaves == 1)
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        else
            lds_barrier();
    };

    // Sums to outputs, in the accumulators' registers.
    const auto finish = [&](int fb, int rb) {
        const rsrc_t rg = make_rsrc(a.w_scales, (uint32_t)a.M * 4u);
        const rsrc_t rs = make_rsrc(a.x_scales + rb, (uint32_t)(a.N - rb) * 4u);
        float sx[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            sx[rt] = __builtin_bit_cast(float, bload4<kAuxCached>(rs, 4 * (wr * RT * 16 + rt * 16 + j), 0));
        const int f0 = fb + wf * FO * 16;
        if constexpr (GATED) {
            const rsrc_t rsu = make_rsrc(a.up_scales, (uint32_t)a.M * 4u);
            const auto all = [&](auto KIND) {
#pragma unroll
                for (int ft = 0; ft < FO; ++ft)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int o = 4 * (f0 + row_w<FO>(ft, 4 * g) + r);
                        const float sg = __builtin_bit_cast(float, bload4<kAuxCached>(rg, o, 0));
                        const float su = __builtin_bit_cast(float, bload4<kAuxCached>(rsu, o, 0));
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const float gate = activate<KIND.value, FINE>((float)acc[ft][rt][r] * sx[rt] * sg);
                            acc[ft][rt][r] =
                                __builtin_bit_cast(int, gate * ((float)acc[ft + FO][rt][r] * sx[rt] * su));
                        }
                    }
            };
            if (a.activation == VQ_ACT_SILU)
                all(std::integral_constant<int, VQ_ACT_SILU>{});
            else if (a.activation == VQ_ACT_GELU)
                all(std::integral_constant<int, VQ_ACT_GELU>{});
            else
                all(std::integral_constant<int, VQ_ACT_GELU_TANH>{});
        } else {
            const bool biased = a.bias != nullptr;
            const rsrc_t rb4 = make_rsrc(biased ? a.bias : a.w_scales, (uint32_t)a.M * 4u);
#pragma unroll
            for (int ft = 0; ft < FT; ++ft)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int o = 4 * (f0 + row_w<FO>(ft, 4 * g) + r);
                    const float sg = __builtin_bit_cast(float, bload4<kAuxCached>(rg, o, 0));
                    // (y + -0 is y: no bias changes no bit)
                    const float add = biased ? __builtin_bit_cast(float, bload4<kAuxCached>(rb4, o, 0)) : -0.0f;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        acc[ft][rt][r] = __builtin_bit_cast(int, __builtin_fmaf((float)acc[ft][rt][r] * sx[rt], sg, add));
                }
        }
    };
    const auto store = [&](int fb, int rb) {
        constexpr int kRun = FO == 1 ? 1 : 2;  // tiles whose values lie side by side in a row
        const int f0 = fb + wf * FO * 16 + row_w<FO>(0, 4 * g), n0 = rb + wr * RT * 16 + j;
        const auto all = [&](auto OD) {
            constexpr int esz = OD.value == VQ_DTYPE_F32 ? 4 : 2, kWords = kRun * esz;
            struct __attribute__((packed, aligned(esz))) Run {  // rows begin where M makes them begin
                uint32_t w[kWords];
            };
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int n = n0 + rt * 16;
                uint8_t *row = static_cast<uint8_t *>(a.out) + ((size_t)n * (size_t)a.M + (size_t)f0) * esz;
                if (n < a.N) {
#pragma unroll
                    for (int q = 0; q < FO / kRun; ++q) {
                        float v[4 * kRun];
#pragma unroll
                        for (int e = 0; e < 4 * kRun; ++e) {
                            const int bits = acc[kRun * q + e / 4][rt][e % 4];  // (a cast of the element reads element 0)
                            v[e] = __builtin_bit_cast(float, bits);
                        }
                        const int left = a.M - (f0 + 32 * q);
                        if (left >= 4 * kRun) {
                            Run o;
#pragma unroll
                            for (int e = 0; e < kWords; ++e) {
                                if constexpr (OD.value == VQ_DTYPE_F32)
                                    o.w[e] = __builtin_bit_cast(uint32_t, v[e]);
                                else if constexpr (OD.value == VQ_DTYPE_BF16)
                                    o.w[e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[2 * e])) |
                                             (uint32_t)__builtin_bit_cast(uint16_t, static_cast<__bf16>(v[2 * e + 1])) << 16;
                                else
                                    o.w[e] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[2 * e])) |
                                             (uint32_t)__builtin_bit_cast(uint16_t, static_cast<_Float16>(v[2 * e + 1])) << 16;
                            }
                            *reinterpret_cast<Run *>(row + 32 * q * esz) = o;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4 * kRun; ++e)
                                if (e < left)
                                    store_out(row, OD.value, 32 * q + e, v[e]);
                        }
                    }
                }
            }
        };
        if (FINE || (!GATED && a.out_dtype == VQ_DTYPE_F32))
            all(std::integral_constant<int, VQ_DTYPE_F32>{});
        else if (a.out_dtype == VQ_DTYPE_BF16)
            all(std::integral_constant<int, VQ_DTYPE_BF16>{});
        else
            all(std::integral_constant<int, VQ_DTYPE_F16>{});
    };

    // A tile cut between workgroups: each stores its sums, agent-coherent and
    // waited for, then counts in; the last adds the others' to its own.  Per
    // wave: the waves of a tile's workgroups hold the same outputs.
    const auto join = [&](const Part &p) -> bool {
        const rsrc_t rp = make_rsrc(reinterpret_cast<uint8_t *>(a.counters) + kCounterBytes,
                                    (uint32_t)(rest * a.cuts) * (uint32_t)kSlot);
        const int t = p.tile - a.whole;
        const auto slot = [&](int cut) { return (cut * rest + t) * kSlot + wave * FT * RT * 1024; };
        const int mine = slot(my_cut);
#pragma unroll
        for (int ft = 0; ft < FT; ++ft)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[ft][rt]), rp,
                                                       16 * lane + (ft * RT + rt) * 1024, mine, kCoherent);
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");
        uint32_t *count = a.counters + t * kWaves + wave;
        uint32_t old = 0;
        if (lane == 0)
            old = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (__builtin_amdgcn_readfirstlane(old) != (uint32_t)(a.cuts - 1))
            return false;
        if (lane == 0)  // every piece has arrived: the counter is ready for the next call
            __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" ::: "memory");
        // so many loads go out together, of kBatch workgroups' pieces or of a part of one
        constexpr int kTiles = FT * RT, kAtOnce = kTiles <= 16 ? kTiles : 8, kBatch = kTiles <= 8 ? 8 / kTiles : 1;
        static_assert(kTiles % kAtOnce == 0, "every tile of a wave is in a batch");
        for (int w0 = 0; w0 < a.cuts; w0 += kBatch) {
            static_for<kTiles / kAtOnce>([&](auto H) {
                u32x4 v[kBatch][kAtOnce];
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const int who = w0 + q;
                    const bool other = who < a.cuts && who != my_cut;
                    const int theirs = other ? slot(who) : 0;
                    const int off = other ? 16 * lane : kOutOfRange;
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e)
                        v[q][e] = __builtin_amdgcn_raw_buffer_load_b128(rp, off + (H.value * kAtOnce + e) * 1024,
                                                                        theirs, kCoherent);
                }
#pragma unroll
                for (int q = 0; q < kBatch; ++q)
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e) {
                        constexpr int t0 = H.value * kAtOnce;
                        acc[(t0 + e) / RT][(t0 + e) % RT] += __builtin_bit_cast(i32x4, v[q][e]);
                    }
            });
        }
        return true;
    };

    // The operands of a step are read while the one before it is multiplied.
    // The barrier comes before a chunk's last step: by then every wave holds
    // the last operands of the chunk, whose stage takes the chunk STAGES ahead,
    // and reads on in the next.
    open();
#pragma unroll 1
    for (int s = 0; s < STAGES; ++s) {
        load(s, std::integral_constant<int, 0>{}, std::integral_constant<int, kMost>{});
        loaded();
    }
    landed(std::integral_constant<int, STAGES - 1>{});
    int stage = 0;
    for (int i = 0; i < parts; ++i) {
        const Part p = part(i);
#pragma unroll
        for (int ft = 0; ft < FT; ++ft)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                acc[ft][rt] = i32x4{0, 0, 0, 0};
        // a part's first operands (again: nothing is held over the end of a part)
#pragma unroll
        for (int ft = 0; ft < FT; ++ft)
            wa[ft] = read_w(0, ft, stage);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            xb[rt] = read_x(0, rt, stage);
        for (int c = p.c0; c < p.c1; ++c) {
            static_for<kSteps>([&](auto S) {
                constexpr bool last = S.value == kSteps - 1;
                const int free = stage;
                if constexpr (last) {
                    landed(std::integral_constant<int, STAGES - 2>{});
                    stage = stage + 1 == STAGES ? 0 : stage + 1;
                }
                constexpr int next = last ? 0 : S.value + 1;
                u32x4 wn[FT];
#pragma unroll
                for (int ft = 0; ft < FT; ++ft)
                    wn[ft] = read_w(next, ft, stage);
                // (the scheduler would sink these reads to their uses)
                __builtin_amdgcn_sched_barrier(0);
                static_for<RT>([&](auto R) {
                    constexpr int rt = R.value;
#pragma unroll
                    for (int ft = 0; ft < FT; ++ft)
                        acc[ft][rt] = mfma_i8(wa[ft], xb[rt], acc[ft][rt]);
                    xb[rt] = read_x(next, rt, stage);
                    // a part of the loads between the matrix instructions: all at
                    // once they fill the address unit's queue and stop the wave
                    if constexpr (last)
                        load(free, std::integral_constant<int, rt * kMost / RT>{},
                             std::integral_constant<int, (rt + 1) * kMost / RT>{});
                    __builtin_amdgcn_sched_barrier(0);
                });
                if constexpr (last)
                    loaded();
#pragma unroll
                for (int ft = 0; ft < FT; ++ft)
                    wa[ft] = wn[ft];
            });
        }
        if constexpr (WK > 1) {
            // the groups' sums, added by the first
            i32x4 *red = reinterpret_cast<i32x4 *>(lds + WK * STAGES * kStage) + wave * FT * RT * 64 + lane;
            constexpr int kGroup = kWaves * FT * RT * 64;
            if (wk > 0)
#pragma unroll
                for (int ft = 0; ft < FT; ++ft)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        red[(wk - 1) * kGroup + (ft * RT + rt) * 64] = acc[ft][rt];
            lds_barrier();
            if (wk == 0)
#pragma unroll
                for (int k = 1; k < WK; ++k)
#pragma unroll
                    for (int ft = 0; ft < FT; ++ft)
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            acc[ft][rt] += red[(k - 1) * kGroup + (ft * RT + rt) * 64];
            lds_barrier();  // read before the next part's are written
            if (wk > 0)
                continue;
        }
        if (p.c1 - p.c0 == nch || join(p)) {
            int fb, rb;
            place(p.tile, fb, rb);
            finish(fb, rb);
            // Loads and stores complete in order: what is in flight is waited
            // for before the stores, so that the next chunks' waits do not
            // wait for these (and the compiler need not for finish's loads).
            wait_vmcnt<0>();
            settled = STAGES - 1;
            store(fb, rb);
        }
    }
    wait_vmcnt<0>();  // loads past the last chunk write LDS: none outlives the workgroup
}

int current_device() {
    int dev = 0;
    return hipGetDevice(&dev) == hipSuccess && dev >= 0 ? dev : 64;
}

// Compute units of a device: the persistent workgroups of a launch, one each.
int device_cus(int dev) {
    static std::atomic<int> known[64];
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (dev >= 64 || hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
            return 256;
        n = std::min(n, kMaxGroups);
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int I, bool GATED, bool FINE, int AUX>
hipError_t launch_form(const W8A8Args &p, const Plan &plan, int dev) {
    constexpr Form f = kForms[I];
    constexpr int BM = f.rows(), BF = f.feats(), kOutFeats = GATED ? BF / 2 : BF;
    constexpr int kLds = f.wk * f.stages * (BF + BM) * KC + (f.wk - 1) * BM * BF * 4;
    static_assert(kLds * f.per_cu <= 160 * 1024, "LDS");
    const auto kern = w8a8_kernel<f.rt, f.ft, f.wr, f.wf, f.wk, f.stages, GATED, FINE, AUX>;
    static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may use that much LDS
    if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (e != hipSuccess)
            return e;
        if (dev < 64)
            allowed.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
    const KArgs a{p.w, p.up, p.x, p.w_scales, p.up_scales, p.x_scales, p.bias, p.out,
                  static_cast<uint32_t *>(p.workspace), p.N, p.M, p.K, p.out_dtype, p.activation,
                  (p.N + BM - 1) / BM, (p.M + kOutFeats - 1) / kOutFeats, plan.whole, plan.cuts};
    hipLaunchKernelGGL(kern, dim3(plan.groups), dim3(64 * f.wr * f.wf * f.wk), kLds, p.stream, a);
    return hipGetLastError();
}

template <bool GATED, int I = 0>
hipError_t launch_plan(const W8A8Args &p, const Plan &plan, int dev) {
    if constexpr (I + 1 < kFormCount)
        if (plan.form != I)
            return launch_plan<GATED, I + 1>(p, plan, dev);
    const bool past = past_caches(kForms[I], p.N, p.M, p.K, GATED);
    if constexpr (GATED)
        if (p.out_dtype == VQ_DTYPE_F32)
            return past ? launch_form<I, true, true, kAuxStream>(p, plan, dev)
                        : launch_form<I, true, true, kAuxCached>(p, plan, dev);
    return past ? launch_form<I, GATED, false, kAuxStream>(p, plan, dev)
                : launch_form<I, GATED, false, kAuxCached>(p, plan, dev);
}

template <bool GATED>
hipError_t launch_rows(W8A8Args p) {
    const int dev = current_device(), cus = device_cus(dev);
    const int most = rows_at_once(p.N, p.M);
    const int N = p.N;
    for (int n0 = 0; n0 < N; n0 += most) {
        W8A8Args part = p;
        part.x += (size_t)n0 * p.K;
        part.x_scales += n0;
        part.out = static_cast<char *>(p.out) + (size_t)n0 * p.M * (p.out_dtype == VQ_DTYPE_F32 ? 4 : 2);
        part.N = std::min(most, N - n0);
        const hipError_t e = launch_plan<GATED>(part, plan_of(part.N, part.M, part.K, GATED, cus, part.workspace ? part.workspace_bytes : 0), dev);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace

size_t w8a8_workspace(int N) {
    const int cus = device_cus(current_device());
    size_t need = 0;
    for (const Form &f : kForms)
        if (fits_rows(f, N))
            need = std::max(need, pieces_bytes(f, cus));
    return need;
}

size_t w8a8_workspace_used(int N, int M, int K, bool gated) {
    const int cus = device_cus(current_device()), most = rows_at_once(N, M);
    const size_t room = w8a8_workspace(N);
    size_t used = 0;
    for (int n : {most, N % most})  // the launches' sizes
        if (n > 0)
            used = std::max(used, plan_bytes(plan_of(n, M, K, gated, cus, room), n, M, gated));
    return used;
}

hipError_t launch_w8a8(const W8A8Args &p) { return p.up ? launch_rows<true>(p) : launch_rows<false>(p); }

}  // namespace vq
