// rotate.hip -- the rotation of queries and keys by their positions.
//
// Pair i of a head (elements i and i + rot / 2, or 2 i and 2 i + 1) turns by
// the angle p f_i, p = ctx_len + the node's depth in its tree.  The angle is
// formed and reduced to a fraction of a turn in 64 bits: at p = 10^6 an fp32
// product alone would be off by up to 2^-24 10^6 = 0.06 of an angle.
//
// One workgroup per token: its rot / 2 sines and cosines once, through LDS, then
// all heads of queries and keys, 16 + 16 bytes (8 pairs) a thread and step.
#include "layer_internal.h"
#include "vq_device.h"

namespace vq {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = VQ_MAX_ROTATE_DIM / 2;

struct KArgs {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
    const float *inv_freq;
    const int32_t *ctx_len;
    const uint64_t *tree_mask;
    int n, q_heads, kv_heads, head_dim, rot_dim;
    float scale;
};

template <bool BF16>
__device__ __forceinline__ void unpack8(u32x4 w, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = BF16 ? __builtin_bit_cast(float, w[e] << 16) : h2f(w[e]);
        v[2 * e + 1] = BF16 ? __builtin_bit_cast(float, w[e] & 0xFFFF0000u) : h2f(w[e] >> 16);
    }
}
template <bool BF16>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint16_t h[2];
#pragma unroll
        for (int o = 0; o < 2; ++o)
            h[o] = BF16 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[2 * e + o]))
                        : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[2 * e + o]));
        w[e] = h[0] | (uint32_t)h[1] << 16;
    }
    return w;
}

template <bool BF16, bool PAIRS>  // PAIRS: neighbouring elements form a pair
__global__ __launch_bounds__(kThreads) void rotate_kernel(KArgs a) {
    __shared__ __attribute__((aligned(16))) float cs[kMaxHalf], sn[kMaxHalf];
    const int64_t row = blockIdx.x;
    const int b = (int)(row / a.n), i = (int)(row - (int64_t)b * a.n);
    const int half = a.rot_dim / 2;
    int64_t pos = max(a.ctx_len[b], 0);
    pos += a.tree_mask ? __popcll(a.tree_mask[row] & (((uint64_t)1 << i) - 1)) : i;
    for (int f = (int)threadIdx.x; f < half; f += kThreads) {
        // turns = p f / (2 pi), its whole part dropped in 64 bits; then
        // sin and cos of pi times twice the rest, |2 rest| <= 1
        const double turns = (double)pos * (double)a.inv_freq[f] * 0.15915494309189533577;
        const float rest = (float)(2.0 * (turns - rint(turns)));
        float s, c;
        sincospif(rest, &s, &c);
        cs[f] = c * a.scale;
        sn[f] = s * a.scale;
    }
    __syncthreads();
    const int per_head = a.head_dim / 16, rot_items = a.rot_dim / 16;
    const int q_items = a.q_heads * per_head, items = q_items + (a.k ? a.kv_heads * per_head : 0);
    for (int t = (int)threadIdx.x; t < items; t += kThreads) {
        const bool key = t >= q_items;
        const int u = key ? t - q_items : t, h = u / per_head, e = u % per_head;
        const int64_t head = (int64_t)h * a.head_dim;
        const uint16_t *src = (key ? a.k + row * a.k_stride : a.q + row * a.q_stride) + head;
        uint16_t *dst = (key ? a.k_out + row * a.k_out_stride : a.q_out + row * a.q_out_stride) + head;
        int lo = 16 * e, hi = lo + 8;
        const bool turn = e < rot_items;
        if (!PAIRS && turn)
            lo = 8 * e, hi = lo + half;
        const u32x4 wl = ld16(src + lo), wh = ld16(src + hi);
        if (!turn) {
            if (dst != src) {
                *reinterpret_cast<u32x4 *>(dst + lo) = wl;
                *reinterpret_cast<u32x4 *>(dst + hi) = wh;
            }
            continue;
        }
        float x[8], y[8], c[8], s[8];
        unpack8<BF16>(wl, x);
        unpack8<BF16>(wh, y);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const f32x4 cv = *reinterpret_cast<const f32x4 *>(cs + 8 * e + 4 * v);
            const f32x4 sv = *reinterpret_cast<const f32x4 *>(sn + 8 * e + 4 * v);
#pragma unroll
            for (int o = 0; o < 4; ++o)
                c[4 * v + o] = cv[o], s[4 * v + o] = sv[o];
        }
        float p[8], r[8];
        if constexpr (PAIRS) {
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                p[2 * o] = x[2 * o] * c[o] - x[2 * o + 1] * s[o];
                p[2 * o + 1] = x[2 * o + 1] * c[o] + x[2 * o] * s[o];
                r[2 * o] = y[2 * o] * c[4 + o] - y[2 * o + 1] * s[4 + o];
                r[2 * o + 1] = y[2 * o + 1] * c[4 + o] + y[2 * o] * s[4 + o];
            }
        } else {
#pragma unroll
            for (int o = 0; o < 8; ++o) {
                p[o] = x[o] * c[o] - y[o] * s[o];
                r[o] = y[o] * c[o] + x[o] * s[o];
            }
        }
        *reinterpret_cast<u32x4 *>(dst + lo) = pack8<BF16>(p);
        *reinterpret_cast<u32x4 *>(dst + hi) = pack8<BF16>(r);
    }
}

}  // namespace

hipError_t launch_rotate(const RotateArgs &p) {
    const KArgs a{static_cast<const uint16_t *>(p.q), static_cast<const uint16_t *>(p.k),
                  static_cast<uint16_t *>(p.q_out), static_cast<uint16_t *>(p.k_out), p.q_stride, p.k_stride,
                  p.q_out_stride, p.k_out_stride, p.inv_freq, p.ctx_len, p.tree_mask, p.n, p.q_heads, p.kv_heads,
                  p.head_dim, p.rot_dim, p.scale};
    const bool bf = p.dtype == VQ_DTYPE_BF16;
    const auto kern = bf ? (p.interleaved ? rotate_kernel<true, true> : rotate_kernel<true, false>)
                         : (p.interleaved ? rotate_kernel<false, true> : rotate_kernel<false, false>);
    hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)p.batch * p.n)), dim3(kThreads), 0, p.stream, a);
    return hipGetLastError();
}

}  // namespace vq
