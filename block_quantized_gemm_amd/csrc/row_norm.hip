// row_norm.hip -- the residual update between two blocks with the norms on
// both sides of it, and the quantization of rows to 8 bits.
//
//   u = y, or post[c] y / sqrt(mean(y^2) + eps)
//   x = residual + alpha gate u          -> residual_out, rounded to its type
//   h = weight[c] x / sqrt(mean(x^2) + eps)   (x before that rounding)
//   out = h in 16 bits, or s = max|h| / 127 and rint(h / s) in 8
//
// One workgroup per row, the row in registers from the first read to the last
// write: every byte moves once.  Sums, x and h are fp32.
#include "layer_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

struct KArgs {
    const void *residual, *y, *gate;
    const float *post_weight, *weight;
    void *residual_out, *out;
    float *scales_out;
    float alpha, eps;
    int C, residual_dtype, y_dtype, out_dtype;
    bool gate_rows, raw;
};

// 8 elements from element index i of a 16-bit or fp32 array
__device__ __forceinline__ void load8(const void *p, int dtype, size_t i, float (&v)[8]) {
    if (dtype == VQ_DTYPE_F32) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + i);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = a[e], v[e + 4] = b[e];
        return;
    }
    const u32x4 w = ld16(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (dtype == VQ_DTYPE_BF16) {
            v[2 * e] = __builtin_bit_cast(float, w[e] << 16);
            v[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
        } else {
            v[2 * e] = h2f(w[e]);
            v[2 * e + 1] = h2f(w[e] >> 16);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int dtype) {
    if (dtype == VQ_DTYPE_BF16)
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
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + i) =
        u32x4{pack2(v[0], v[1], dtype), pack2(v[2], v[3], dtype), pack2(v[4], v[5], dtype), pack2(v[6], v[7], dtype)};
}

// Sum (or maximum) over the workgroup, the same bits in every thread.
template <bool MAX>
__device__ __forceinline__ float reduce(float v, float *lds) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const float o = __shfl_xor(v, d);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    const int waves = (int)blockDim.x >> 6;
    if (waves == 1)
        return v;
    __syncthreads();  // the values of an earlier reduction have been read
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float r = lds[0];
    for (int w = 1; w < waves; ++w)
        r = MAX ? fmaxf(r, lds[w]) : r + lds[w];
    return r;
}

// VPT: vectors of 8 elements a thread holds
template <int VPT>
__global__ __launch_bounds__(1024) void row_norm_kernel(KArgs a) {
    __shared__ float lds[16];
    const int vecs = a.C / 8;
    const size_t row = (size_t)blockIdx.x * a.C;
    float x[VPT][8];
    bool in[VPT];
    int at[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = (int)(threadIdx.x + i * blockDim.x);
        in[i] = v < vecs;
        at[i] = 8 * v;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[i][e] = 0.f;
        if (in[i])
            load8(a.residual, a.residual_dtype, row + at[i], x[i]);
    }
    if (a.y) {
        float y[VPT][8];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[i][e] = 0.f;
            if (in[i])
                load8(a.y, a.y_dtype, row + at[i], y[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = __builtin_fmaf(y[i][e], y[i][e], sum);
        }
        const float inv = a.post_weight ? 1.0f / sqrtf(reduce<false>(sum, lds) / (float)a.C + a.eps) : 1.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!in[i])
                continue;
            float t[8];
            if (a.post_weight) {
                load8(a.post_weight, VQ_DTYPE_F32, at[i], t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[i][e] = y[i][e] * inv * t[e];
            }
            if (a.gate) {
                if (a.gate_rows)
                    load8(a.gate, a.y_dtype, row + at[i], t);
                else
                    load8(a.gate, VQ_DTYPE_F32, at[i], t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[i][e] *= t[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[i][e] = __builtin_fmaf(a.alpha, y[i][e], x[i][e]);
            if (a.residual_out)
                store8(a.residual_out, a.residual_dtype, row + at[i], x[i]);
        }
    }
    if (!a.raw) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = __builtin_fmaf(x[i][e], x[i][e], sum);
        const float inv = 1.0f / sqrtf(reduce<false>(sum, lds) / (float)a.C + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float t[8];
            if (a.weight && in[i]) {
                load8(a.weight, VQ_DTYPE_F32, at[i], t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[i][e] = x[i][e] * inv * t[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[i][e] *= inv;
            }
        }
    }
    if (a.out_dtype != VQ_DTYPE_I8) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (in[i])
                store8(a.out, a.out_dtype, row + at[i], x[i]);
        return;
    }
    // A NaN or an infinity anywhere in the row makes the scale NaN and every
    // code 0, so that it shows in what is computed from the row.
    float top = 0.f, bad = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float m = fabsf(x[i][e]);
            top = fmaxf(top, m);
            bad = m < __builtin_inff() ? bad : 1.f;
        }
    top = reduce<true>(bad > 0.f ? __builtin_inff() : top, lds);
    const bool ok = top < __builtin_inff();
    const float s = top / 127.0f;
    if (threadIdx.x == 0)
        a.scales_out[blockIdx.x] = ok ? s : __builtin_nanf("");
    int8_t *out = static_cast<int8_t *>(a.out) + row;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (!in[i])
            continue;
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = ok && s > 0.f ? fminf(fmaxf(rintf(x[i][e] / s), -127.f), 127.f) : 0.f;
            w[e >> 2] |= ((uint32_t)(int)q & 0xFFu) << (8 * (e & 3));
        }
        *reinterpret_cast<u32x2 *>(out + at[i]) = u32x2{w[0], w[1]};
    }
}

}  // namespace

hipError_t launch_row_norm(const RowNormArgs &p) {
    const int vecs = p.C / 8;
    const int vpt = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    const int threads = ((vecs + vpt - 1) / vpt + 63) / 64 * 64;
    const KArgs a{p.residual, p.y, p.gate, p.post_weight, p.weight, p.residual_out, p.out, p.scales_out, p.alpha,
                  p.eps, p.C, p.residual_dtype, p.y_dtype, p.out_dtype, p.gate_rows, p.raw};
    const auto kern = vpt == 1 ? row_norm_kernel<1> : vpt == 2 ? row_norm_kernel<2> : row_norm_kernel<4>;
    // a grid dimension holds 2^32 - 1 threads
    constexpr int kRows = 1 << 21;
    for (int r0 = 0; r0 < p.N; r0 += kRows) {
        KArgs b = a;
        const size_t at = (size_t)r0 * p.C;
        const auto skip = [&](const void *q, int dtype) {
            return q ? static_cast<const char *>(q) + at * (dtype == VQ_DTYPE_F32 ? 4 : dtype == VQ_DTYPE_I8 ? 1 : 2)
                     : nullptr;
        };
        b.residual = skip(p.residual, p.residual_dtype);
        b.y = skip(p.y, p.y_dtype);
        if (p.gate_rows)
            b.gate = skip(p.gate, p.y_dtype);
        b.residual_out = const_cast<char *>(skip(p.residual_out, p.residual_dtype));
        b.out = const_cast<char *>(skip(p.out, p.out_dtype));
        b.scales_out = p.scales_out ? p.scales_out + r0 : nullptr;
        hipLaunchKernelGGL(kern, dim3(std::min(kRows, p.N - r0)), dim3(threads), 0, p.stream, b);
    }
    return hipGetLastError();
}

}  // namespace vq
