// row_norm.hip -- the residual update between two blocks with the norms on
// both sides of it, and the quantization of rows to 8 bits.
//
//   u = y, or post[c] y / sqrt(mean(y^2) + eps)
//   x = residual + alpha gate u          -> residual_out, rounded to its type
//   h = weight[c] x / sqrt(mean(x^2) + eps)   (x before that rounding)
//   out = h in 16 bits, or s = max|h| / 127 and rint(h / s) in 8
//
// One workgroup per row, the row in registers from the first read to the last
// write: every byte moves once.  All of a thread's loads are issued before any
// value is used (with the conversion beside each load they came one after the
// other).  Sums, x and h are fp32.
#include "layer_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// 8 elements as they lie in memory
template <bool WIDE>
struct Raw {
    u32x4 v[WIDE ? 2 : 1];
};
template <bool WIDE>
__device__ __forceinline__ Raw<WIDE> load8(const void *p, size_t i) {
    Raw<WIDE> r;
    const u32x4 *q = reinterpret_cast<const u32x4 *>(static_cast<const char *>(p) + i * (WIDE ? 4 : 2));
    r.v[0] = q[0];
    if constexpr (WIDE)
        r.v[1] = q[1];
    return r;
}
template <bool WIDE>
__device__ __forceinline__ void to_float(const Raw<WIDE> &r, bool bf16, float (&v)[8]) {
    if constexpr (WIDE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t bits = r.v[e / 4][e % 4];
            v[e] = __builtin_bit_cast(float, bits);
        }
    } else if (bf16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __builtin_bit_cast(float, r.v[0][e] << 16);
            v[2 * e + 1] = __builtin_bit_cast(float, r.v[0][e] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = h2f(r.v[0][e]);
            v[2 * e + 1] = h2f(r.v[0][e] >> 16);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool bf16) {
    if (bf16)
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(lo)) |
               (uint32_t)__builtin_bit_cast(uint16_t, static_cast<__bf16>(hi)) << 16;
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(lo)) |
           (uint32_t)__builtin_bit_cast(uint16_t, static_cast<_Float16>(hi)) << 16;
}
__device__ __forceinline__ void store8(void *p, int dtype, size_t i, const float (&v)[8]) {
    if (dtype == VQ_DTYPE_F32) {
        f32x4 *q = reinterpret_cast<f32x4 *>(static_cast<float *>(p) + i);
        q[0] = f32x4{v[0], v[1], v[2], v[3]};
        q[1] = f32x4{v[4], v[5], v[6], v[7]};
        return;
    }
    const bool bf = dtype == VQ_DTYPE_BF16;
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + i) =
        u32x4{pack2(v[0], v[1], bf), pack2(v[2], v[3], bf), pack2(v[4], v[5], bf), pack2(v[6], v[7], bf)};
}

// Reduction over the workgroup, the same bits in every thread.
template <typename T, typename F>
__device__ __forceinline__ T reduce(T v, T *lds, F &&f) {
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v = f(v, __shfl_xor(v, d));
    const int waves = (int)blockDim.x >> 6;
    if (waves == 1)
        return v;
    __syncthreads();  // the values of an earlier reduction have been read
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    T r = lds[0];
    for (int w = 1; w < waves; ++w)
        r = f(r, lds[w]);
    return r;
}

// Bits of |v|: as integers they order like the values, infinity and NaN last.
constexpr uint32_t kInfBits = 0x7F800000u;
__device__ __forceinline__ uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

// The scale of a row whose largest magnitude has these bits, and what its
// codes need.
struct Scale {
    float s, inv;
    int how;  // 0: codes 0, 1: quotients from the reciprocal, 2: divisions
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {
    if (top >= kInfBits)  // an infinity or a NaN somewhere in the row
        return Scale{__builtin_nanf(""), 0.f, 0};
    const float s = __builtin_bit_cast(float, top) / 127.0f;
    if (!(s > 0.f))
        return Scale{s, 0.f, 0};
    return Scale{s, 1.0f / s, s >= 0x1p-90f && s <= 0x1p90f ? 1 : 2};
}
// Codes of 8 values.  x / s correctly rounded without a division: inv is the
// correctly rounded reciprocal, the first product is refined to within a unit
// of the quotient, and one more step from there gives its correct rounding
// (every residual is exact by FMA where s is far from the ends of the range;
// else divisions).  Adding 1.5 2^23 rounds to the nearest integer, halves to
// even, and leaves it in the low bits.  |x / s| <= 127 (1 + 2^-23): no clamp.
// Divisions alone took 98 us of 4,093 rows of 17,408; this way 41.
__device__ __forceinline__ u32x2 codes8(const float (&x)[8], const Scale &k) {
    if (k.how == 0)
        return u32x2{0u, 0u};
    uint32_t q[8];
    if (k.how == 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q0 = x[e] * k.inv;
            const float q1 = __builtin_fmaf(__builtin_fmaf(-q0, k.s, x[e]), k.inv, q0);
            const float q2 = __builtin_fmaf(__builtin_fmaf(-q1, k.s, x[e]), k.inv, q1);
            q[e] = __builtin_bit_cast(uint32_t, q2 + 12582912.0f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = (uint32_t)(int)fminf(fmaxf(rintf(x[e] / k.s), -127.f), 127.f);
    }
    u32x2 w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __builtin_amdgcn_perm(q[4 * h + 1], q[4 * h], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(q[4 * h + 3], q[4 * h + 2], 0x04000C0Cu);
        w[h] = lo | hi;
    }
    return w;
}

struct KArgs {
    const void *residual, *y, *gate;
    const float *post_weight, *weight;
    void *residual_out, *out;
    float *scales_out;
    float alpha, eps;
    int C, residual_dtype, y_dtype, out_dtype;
    bool gate_rows;
};

// VPT: vectors of 8 elements a thread holds; WIDE: an fp32 residual
template <int VPT, bool WIDE>
__global__ __launch_bounds__(1024) void row_norm_kernel(KArgs a) {
    __shared__ float lds[16];
    const auto sum_of = [](float p, float q) { return p + q; };
    const int vecs = a.C / 8;
    const size_t row = (size_t)blockIdx.x * a.C;
    const bool y_bf = a.y_dtype == VQ_DTYPE_BF16;
    bool in[VPT];
    int at[VPT];
    Raw<WIDE> rr[VPT];
    Raw<false> ry[VPT], rg[VPT];
    const bool gated_rows = a.gate && a.gate_rows;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = (int)(threadIdx.x + i * blockDim.x);
        in[i] = v < vecs;
        at[i] = 8 * (in[i] ? v : 0);
        rr[i] = load8<WIDE>(a.residual, row + at[i]);
        if (a.y)
            ry[i] = load8<false>(a.y, row + at[i]);
        if (gated_rows)
            rg[i] = load8<false>(a.gate, row + at[i]);
    }
    // 1 / sqrt(mean(v^2) + eps).  Where that mean is below 2^-90 or infinite, so
    // that squares may have left fp32's range, v is multiplied by a power of two
    // first and stays so: v times the result is what it would be.
    const auto inverse_rms = [&](float (&v)[VPT][8]) {
        const auto mean = [&] {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i])
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum = __builtin_fmaf(v[i][e], v[i][e], sum);
            return reduce(sum, lds, sum_of) / (float)a.C;
        };
        float m = mean() + a.eps;
        if (!(m >= 0x1p-90f && m <= 3.4028235e38f)) {  // (the same bits in every thread)
            const float s = m < 1.0f ? 0x1p100f : 0x1p-100f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[i][e] *= s;
            m = mean() + a.eps * s * s;
        }
        return 1.0f / sqrtf(m);
    };
    float x[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        to_float<WIDE>(rr[i], a.residual_dtype == VQ_DTYPE_BF16, x[i]);
    if (a.y) {
        float y[VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            to_float<false>(ry[i], y_bf, y[i]);
        const float inv = a.post_weight ? inverse_rms(y) : 1.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float t[8];
            if (a.post_weight) {
                to_float<true>(load8<true>(a.post_weight, at[i]), false, t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[i][e] = y[i][e] * inv * t[e];
            }
            if (a.gate) {
                if (a.gate_rows)
                    to_float<false>(rg[i], y_bf, t);
                else
                    to_float<true>(load8<true>(a.gate, at[i]), false, t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[i][e] *= t[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[i][e] = __builtin_fmaf(a.alpha, y[i][e], x[i][e]);
            if (a.residual_out && in[i])
                store8(a.residual_out, a.residual_dtype, row + at[i], x[i]);
        }
    }
    const float inv = inverse_rms(x);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float t[8];
        if (a.weight) {
            to_float<true>(load8<true>(a.weight, at[i]), false, t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[i][e] = x[i][e] * inv * t[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[i][e] *= inv;
        }
    }
    if (a.out_dtype != VQ_DTYPE_I8) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in[i])
                store8(a.out, a.out_dtype, row + at[i], x[i]);
        return;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (in[i])
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top = max(top, abs_bits(x[i][e]));
    const Scale k =
        scale_of(reduce(top, reinterpret_cast<uint32_t *>(lds), [](uint32_t p, uint32_t q) { return max(p, q); }));
    if (threadIdx.x == 0)
        a.scales_out[blockIdx.x] = k.s;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (in[i])
            *reinterpret_cast<u32x2 *>(static_cast<int8_t *>(a.out) + row + at[i]) = codes8(x[i], k);
}

// Rows as they are.  The maximum of 16-bit rows is taken on their bits, two
// elements an instruction.
template <int VPT, bool WIDE>
__global__ __launch_bounds__(1024) void row_quant_kernel(const void *__restrict__ x, int dtype,
                                                         int8_t *__restrict__ out, float *__restrict__ scales, int C) {
    __shared__ uint32_t lds[16];
    const auto larger = [](uint32_t p, uint32_t q) { return max(p, q); };
    const int vecs = C / 8;
    const size_t row = (size_t)blockIdx.x * C;
    const bool bf = dtype == VQ_DTYPE_BF16;
    Raw<WIDE> r[VPT];
    bool in[VPT];
    int at[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = (int)(threadIdx.x + i * blockDim.x);
        in[i] = v < vecs;
        at[i] = 8 * (in[i] ? v : 0);  // (a vector of the row twice changes no maximum)
        r[i] = load8<WIDE>(x, row + at[i]);
    }
    uint32_t top = 0;
    if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top = max(top, r[i].v[e / 4][e % 4] & 0x7FFFFFFFu);
        top = reduce(top, lds, larger);
    } else {
        u16x2 most = {0, 0};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t bits = r[i].v[0][e] & 0x7FFF7FFFu;
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, bits));
            }
        top = reduce((uint32_t)max(most[0], most[1]), lds, larger);
        if (bf)
            top <<= 16;
        else  // (fp16's infinity and NaN bits become fp32's)
            top = top >= 0x7C00u ? kInfBits : __builtin_bit_cast(uint32_t, h2f(top));
    }
    const Scale k = scale_of(top);
    if (threadIdx.x == 0)
        scales[blockIdx.x] = k.s;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (in[i]) {
            float v[8];
            to_float<WIDE>(r[i], bf, v);
            *reinterpret_cast<u32x2 *>(out + row + at[i]) = codes8(v, k);
        }
}

// Threads of a workgroup and vectors of each, for rows of C elements.
struct Fit {
    int threads, vpt;
};
// The quantizer, whose threads have little else to do than wait for their
// loads and for each other, is faster with fewer of them a row (8,000 rows of
// 5,120: 25 us with two vectors each, 36 with one; of 8,192: 37, 53); the norm,
// with more registers a vector, is not (8,190 rows of 5,120: 105, 102).
Fit fit(int C, int ones) {
    const int vecs = C / 8, vpt = vecs <= ones ? 1 : vecs <= std::max(1024, 2 * ones) ? 2 : 4;
    return Fit{((vecs + vpt - 1) / vpt + 63) / 64 * 64, vpt};
}
constexpr int kRows = 1 << 21;  // rows per launch: a grid dimension holds 2^32 - 1 threads

template <typename K>
K *skip(K *p, size_t elements, int dtype) {
    using B = std::conditional_t<std::is_const_v<K>, const char, char>;
    return p ? static_cast<B *>(p) + elements * (dtype == VQ_DTYPE_F32 ? 4 : dtype == VQ_DTYPE_I8 ? 1 : 2) : nullptr;
}

}  // namespace

hipError_t launch_row_norm(const RowNormArgs &p) {
    const Fit f = fit(p.C, 1024);
    const bool wide = p.residual_dtype == VQ_DTYPE_F32;
    const auto kern = f.vpt == 1   ? (wide ? row_norm_kernel<1, true> : row_norm_kernel<1, false>)
                      : f.vpt == 2 ? (wide ? row_norm_kernel<2, true> : row_norm_kernel<2, false>)
                                   : (wide ? row_norm_kernel<4, true> : row_norm_kernel<4, false>);
    for (int r0 = 0; r0 < p.N; r0 += kRows) {
        const size_t at = (size_t)r0 * p.C;
        const KArgs a{skip(p.residual, at, p.residual_dtype), skip(p.y, at, p.y_dtype),
                      p.gate_rows ? skip(p.gate, at, p.y_dtype) : p.gate, p.post_weight, p.weight,
                      skip(p.residual_out, at, p.residual_dtype), skip(p.out, at, p.out_dtype),
                      p.scales_out ? p.scales_out + r0 : nullptr, p.alpha, p.eps, p.C, p.residual_dtype, p.y_dtype,
                      p.out_dtype, p.gate_rows};
        hipLaunchKernelGGL(kern, dim3(std::min(kRows, p.N - r0)), dim3(f.threads), 0, p.stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_row_quant(const void *x, int x_dtype, int8_t *q, float *scales, int N, int C, hipStream_t stream) {
    const Fit f = fit(C, 256);
    const bool wide = x_dtype == VQ_DTYPE_F32;
    const auto kern = f.vpt == 1   ? (wide ? row_quant_kernel<1, true> : row_quant_kernel<1, false>)
                      : f.vpt == 2 ? (wide ? row_quant_kernel<2, true> : row_quant_kernel<2, false>)
                                   : (wide ? row_quant_kernel<4, true> : row_quant_kernel<4, false>);
    for (int r0 = 0; r0 < N; r0 += kRows) {
        const size_t at = (size_t)r0 * C;
        hipLaunchKernelGGL(kern, dim3(std::min(kRows, N - r0)), dim3(f.threads), 0, stream, skip(x, at, x_dtype),
                           x_dtype, q + at, scales + r0, C);
    }
    return hipGetLastError();
}

}  // namespace vq
