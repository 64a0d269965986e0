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
// weights as the first operand: a lane then holds 4 consecutive features of
// one row, and in the gated form gate and up of the same feature.  Chunks of
// 128 k are loaded straight into LDS, `STAGES - 1` chunks ahead; 16-byte pieces
// are XOR-swizzled by row so that the operand reads of 16 rows cover all 64
// banks.
#include "layer_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kChunk = 128;            // k per chunk: one 128-byte line of a row
constexpr int kOutOfRange = 0x7FFFFFF0;  // past every range below: the load returns zeros

struct KArgs {
    const int8_t *w, *up, *x;
    const float *w_scales, *up_scales, *x_scales, *bias;
    void *out;
    int N, M, K, out_dtype, activation, row_tiles;
};

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0,
                                                 0);
}

// The activations are written so that no large term is subtracted from
// another: 0.5 g (1 + tanh z) = g / (1 + exp(-2 z)), and the Gaussian's
// distribution function as 0.5 erfc(-g / sqrt 2).
__device__ __forceinline__ float activate(float g, int kind) {
    if (kind == VQ_ACT_SILU)
        return g / (1.0f + expf(-g));
    if (kind == VQ_ACT_GELU_TANH) {
        const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
        return g / (1.0f + expf(-2.0f * z));
    }
    return 0.5f * g * erfcf(g * -0.7071067811865476f);
}

template <int RT, int FT, int WR, int WF, int STAGES, bool GATED>
__global__ __launch_bounds__(64 * WR * WF) void w8a8_kernel(KArgs a) {
    constexpr int kWaves = WR * WF, BM = 16 * RT * WR, BF = 16 * FT * WF;
    constexpr int kWPieces = BF / 8, kPieces = kWPieces + BM / 8;  // 1 KiB each: 8 rows x 128 B
    constexpr int kPer = kPieces / kWaves, kExtra = kPieces % kWaves, kMost = kPer + (kExtra ? 1 : 0);
    constexpr int kStage = kPieces * 1024;
    constexpr int kOutFeats = GATED ? BF / 2 : BF;  // output features of the workgroup
    constexpr int FO = GATED ? FT / 2 : FT;         // output feature tiles of a wave
    static_assert(kWaves % 2 == 0 && (!GATED || FT % 2 == 0), "shape");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = wave_id(), j = lane & 15, g = lane >> 4;
    const int wr = wave % WR, wf = wave / WR;
    const int tile = xcd_run_index((int)blockIdx.x, (int)gridDim.x);
    const int fb = tile / a.row_tiles * kOutFeats, rb = tile % a.row_tiles * BM;
    const int K = a.K, nch = (K + kChunk - 1) / kChunk;

    const int rows = min(BM, a.N - rb), feats = min(kOutFeats, a.M - fb);
    const rsrc_t rx = make_rsrc(a.x + (size_t)rb * K, (uint32_t)rows * (uint32_t)K);
    const rsrc_t rw = make_rsrc(a.w + (size_t)fb * K, (uint32_t)feats * (uint32_t)K);
    const rsrc_t ru = GATED ? make_rsrc(a.up + (size_t)fb * K, (uint32_t)feats * (uint32_t)K) : rw;
    // row 8 p + lane / 8 of a piece p = wave + kWaves i, its 16-byte slot lane % 8:
    // the slot holds the row's bytes 16 (slot ^ (row / 2 % 8)) .. +16
    const int byte16 = 16 * ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
    const int voff = (lane >> 3) * K + byte16;

    auto issue = [&](int c, int stage) {
        const int k0 = c * kChunk;
        // past K the row's neighbour would be read: the activations are
        // zeros there, and so is the product
        const int xoff = k0 + byte16 < K ? voff : kOutOfRange;
        const int woff = c < nch ? voff : kOutOfRange;
        uint8_t *st = lds + stage * kStage;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int p = wave + kWaves * i;
            if (kExtra && i == kMost - 1 && p >= kPieces)
                break;
            if (p >= kWPieces)
                bload16_lds(rx, st + 1024 * p, xoff, 8 * (p - kWPieces) * K + k0);
            else if (GATED && p >= kWPieces / 2)
                bload16_lds(ru, st + 1024 * p, woff, 8 * (p - kWPieces / 2) * K + k0);
            else
                bload16_lds(rw, st + 1024 * p, woff, 8 * p * K + k0);
        }
    };

    i32x4 acc[FT][RT];
#pragma unroll
    for (int ft = 0; ft < FT; ++ft)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            acc[ft][rt] = i32x4{0, 0, 0, 0};

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        issue(s, s);
    const int sw = (j >> 1) & 7;
    int stage = 0;
    for (int c = 0; c < nch; ++c) {
        // all but the newest STAGES - 2 chunks' loads have landed
        if (!kExtra || wave >= kExtra)
            wait_vmcnt<(STAGES - 2) * kPer>();
        else
            wait_vmcnt<(STAGES - 2) * kMost>();
        lds_barrier();  // chunk c is whole, and every wave is done with chunk c - 1
        issue(c + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
        const uint8_t *st = lds + stage * kStage;
        const uint8_t *xs = st + kWPieces * 1024 + (wr * RT * 16 + j) * 128;
        const uint8_t *wl = st + (wf * FO * 16 + j) * 128;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int at = 16 * ((4 * s + g) ^ sw);
            u32x4 xb[RT], wa[FT];
#pragma unroll
            for (int ft = 0; ft < FT; ++ft)
                wa[ft] = *reinterpret_cast<const u32x4 *>(
                    wl + (ft < FO ? ft * 16 : BF / 2 + (ft - FO) * 16) * 128 + at);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                xb[rt] = *reinterpret_cast<const u32x4 *>(xs + rt * 16 * 128 + at);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int ft = 0; ft < FT; ++ft)
                    acc[ft][rt] = mfma_i8(wa[ft], xb[rt], acc[ft][rt]);
        }
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    wait_vmcnt<0>();  // the loads past the last chunk write LDS: none outlives the workgroup

    const size_t M = (size_t)a.M;
    const bool vec = a.M % 4 == 0;
#pragma unroll
    for (int ft = 0; ft < FO; ++ft) {
        const int f = fb + wf * FO * 16 + ft * 16 + 4 * g;
        float sg[4], su[4], add[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool in = f + r < a.M;
            sg[r] = in ? a.w_scales[f + r] : 0.f;
            su[r] = GATED && in ? a.up_scales[f + r] : 0.f;
            add[r] = !GATED && a.bias && in ? a.bias[f + r] : 0.f;
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int n = rb + wr * RT * 16 + rt * 16 + j;
            if (n >= a.N)
                continue;
            const float sx = a.x_scales[n];
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float y = (float)acc[ft][rt][r] * sx * sg[r];
                if constexpr (GATED)
                    v[r] = activate(y, a.activation) * ((float)acc[ft + FO][rt][r] * sx * su[r]);
                else
                    v[r] = a.bias ? y + add[r] : y;
            }
            const size_t at = (size_t)n * M + (size_t)f;
            if (vec && f < a.M) {
                if (a.out_dtype == VQ_DTYPE_F32)
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at) = f32x4{v[0], v[1], v[2], v[3]};
                else {
                    uint16_t h[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        h[r] = a.out_dtype == VQ_DTYPE_BF16
                                   ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[r]))
                                   : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[r]));
                    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + at) =
                        u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (f + r < a.M)
                        store_out(a.out, a.out_dtype, at + r, v[r]);
            }
        }
    }
}

template <int RT, int FT, int WR, int WF, int STAGES, bool GATED>
hipError_t launch_shape(const W8A8Args &p) {
    constexpr int BM = 16 * RT * WR, BF = 16 * FT * WF, kOutFeats = GATED ? BF / 2 : BF;
    constexpr int kLds = STAGES * (BF + BM) * 128;
    const auto kern = w8a8_kernel<RT, FT, WR, WF, STAGES, GATED>;
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess)
        return e;
    const int cols = (p.M + kOutFeats - 1) / kOutFeats, row_tiles = (p.N + BM - 1) / BM;
    const int per_launch = std::max(1, (1 << 22) / cols);  // row tiles per launch: a grid holds 2^32 - 1 threads
    for (int r0 = 0; r0 < row_tiles; r0 += per_launch) {
        const int rt = std::min(per_launch, row_tiles - r0);
        KArgs a{p.w, p.up, p.x + (size_t)r0 * BM * p.K, p.w_scales, p.up_scales, p.x_scales + (size_t)r0 * BM, p.bias,
                static_cast<char *>(p.out) + (size_t)r0 * BM * p.M * (p.out_dtype == VQ_DTYPE_F32 ? 4 : 2),
                std::min(p.N - r0 * BM, rt * BM), p.M, p.K, p.out_dtype, p.activation, rt};
        hipLaunchKernelGGL(kern, dim3(cols * rt), dim3(64 * WR * WF), kLds, p.stream, a);
    }
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_rows(const W8A8Args &p) {
    if (p.N <= 16)
        return launch_shape<1, 2, 1, 4, 6, GATED>(p);
    if (p.N <= 64)
        return launch_shape<4, 2, 1, 4, 4, GATED>(p);
    return launch_shape<8, 4, 2, 4, 2, GATED>(p);
}

}  // namespace

size_t w8a8_workspace(bool gated, int M, int K) {
    (void)gated, (void)M, (void)K;
    return 0;
}

hipError_t launch_w8a8(const W8A8Args &p) { return p.up ? launch_rows<true>(p) : launch_rows<false>(p); }

}  // namespace vq
