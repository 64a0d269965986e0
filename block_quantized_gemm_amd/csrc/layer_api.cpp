// layer_api.cpp -- the C ABI of the decoder-layer operators: argument
// validation and dispatch, under the conventions of vq.h (every argument is
// checked before the first HIP call; on any error nothing is enqueued).
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "layer_internal.h"
#include "vq.h"

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_dev_ok[kMaxDevices];  // 0 unknown, 1 gfx950, 2 other

int check_device() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0)
        return VQ_ERR_DEVICE;
    const int known = dev < kMaxDevices ? g_dev_ok[dev].load(std::memory_order_relaxed) : 0;
    if (known)
        return known == 1 ? VQ_OK : VQ_ERR_DEVICE;
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return VQ_ERR_DEVICE;
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < kMaxDevices)
        g_dev_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
    return ok ? VQ_OK : VQ_ERR_DEVICE;
}

bool aligned(std::initializer_list<const void *> ps, uintptr_t to) {
    for (const void *p : ps)
        if (reinterpret_cast<uintptr_t>(p) & (to - 1))
            return false;
    return true;
}
bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }
bool half_type(int d) { return d == VQ_DTYPE_F16 || d == VQ_DTYPE_BF16; }
bool float_type(int d) { return half_type(d) || d == VQ_DTYPE_F32; }
bool product_ok(int64_t m, int64_t k) {
    return in(m, 1, VQ_MAX_DIM) && in(k, 16, VQ_MAX_W8A8_K) && k % 16 == 0;
}
int status(hipError_t e) { return e == hipSuccess ? VQ_OK : VQ_ERR_LAUNCH; }

int run_product(const vq::W8A8Args &a, int64_t n, int64_t m, int64_t k) {
    if (!float_type(a.out_dtype))
        return VQ_ERR_BAD_DTYPE;
    if (!in(n, 1, VQ_MAX_DIM) || !product_ok(m, k))
        return VQ_ERR_BAD_SHAPE;
    if (!aligned({a.w, a.up, a.x, a.out, a.workspace}, 16) ||
        !aligned({a.w_scales, a.up_scales, a.x_scales, a.bias}, 4))
        return VQ_ERR_MISALIGNED;
    const int dev = check_device();
    if (dev != VQ_OK)
        return dev;
    return status(vq::launch_w8a8(a));
}

}  // namespace

extern "C" {

size_t vq_w8a8_workspace_bytes(int64_t n_rows) {
    return in(n_rows, 1, VQ_MAX_DIM) ? vq::w8a8_workspace((int)n_rows) : 0;
}

size_t vq_w8a8_workspace_used(int64_t n_rows, int64_t m, int64_t k, int gated) {
    return in(n_rows, 1, VQ_MAX_DIM) && product_ok(m, k)
               ? vq::w8a8_workspace_used((int)n_rows, (int)m, (int)k, gated != 0)
               : 0;
}

int vq_gemm_w8a8(const int8_t *w, const float *w_scales, const int8_t *x, const float *x_scales, const float *bias,
                 void *out, int out_dtype, int64_t n_rows, int64_t m, int64_t k, void *workspace,
                 size_t workspace_bytes, void *stream) {
    if (!w || !w_scales || !x || !x_scales || !out)
        return VQ_ERR_NULL_POINTER;
    return run_product({w, nullptr, w_scales, nullptr, x, x_scales, bias, 0, out, out_dtype, (int)n_rows, (int)m,
                        (int)k, workspace, workspace_bytes, static_cast<hipStream_t>(stream)},
                       n_rows, m, k);
}

int vq_gated_w8a8(const int8_t *w_gate, const float *gate_scales, const int8_t *w_up, const float *up_scales,
                  const int8_t *x, const float *x_scales, int activation, void *out, int out_dtype, int64_t n_rows,
                  int64_t f, int64_t k, void *workspace, size_t workspace_bytes, void *stream) {
    if (!w_gate || !gate_scales || !w_up || !up_scales || !x || !x_scales || !out)
        return VQ_ERR_NULL_POINTER;
    if (activation != VQ_ACT_SILU && activation != VQ_ACT_GELU && activation != VQ_ACT_GELU_TANH)
        return VQ_ERR_BAD_CONFIG;
    return run_product({w_gate, w_up, gate_scales, up_scales, x, x_scales, nullptr, activation, out, out_dtype,
                        (int)n_rows, (int)f, (int)k, workspace, workspace_bytes, static_cast<hipStream_t>(stream)},
                       n_rows, f, k);
}

int vq_residual_norm(const void *residual, int residual_dtype, const void *y, int y_dtype, const float *post_weight,
                     const void *gate, int gate_rows, float alpha, const float *weight, float eps,
                     void *residual_out, void *out, int out_dtype, float *scales_out, int64_t n_rows, int64_t c,
                     void *stream) {
    if (!residual || !out || (out_dtype == VQ_DTYPE_I8 && !scales_out))
        return VQ_ERR_NULL_POINTER;
    if (!float_type(residual_dtype) || (y && !half_type(y_dtype)) ||
        (!half_type(out_dtype) && out_dtype != VQ_DTYPE_I8) || (out_dtype != VQ_DTYPE_I8 && scales_out))
        return VQ_ERR_BAD_DTYPE;
    if (!in(n_rows, 1, VQ_MAX_DIM) || !in(c, 16, VQ_MAX_ROW) || c % 16)
        return VQ_ERR_BAD_SHAPE;
    if (!y && (post_weight || gate || residual_out))  // there is no update to apply them to
        return VQ_ERR_BAD_CONFIG;
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return VQ_ERR_BAD_CONFIG;
    if (!aligned({residual, y, post_weight, gate, weight, residual_out, out}, 16) || !aligned({scales_out}, 4))
        return VQ_ERR_MISALIGNED;
    const int dev = check_device();
    if (dev != VQ_OK)
        return dev;
    return status(vq::launch_row_norm({residual, residual_dtype, y, y_dtype, post_weight, gate, gate_rows != 0, alpha,
                                       weight, eps, residual_out, out, out_dtype, scales_out, (int)n_rows,
                                       (int)c, static_cast<hipStream_t>(stream)}));
}

int vq_quant_rows_int8(const void *x, int x_dtype, int8_t *q_out, float *scales_out, int64_t n_rows, int64_t k,
                       void *stream) {
    if (!x || !q_out || !scales_out)
        return VQ_ERR_NULL_POINTER;
    if (!float_type(x_dtype))
        return VQ_ERR_BAD_DTYPE;
    if (!in(n_rows, 1, VQ_MAX_DIM) || !in(k, 16, VQ_MAX_ROW) || k % 16)
        return VQ_ERR_BAD_SHAPE;
    if (!aligned({x, q_out}, 16) || !aligned({scales_out}, 4))
        return VQ_ERR_MISALIGNED;
    const int dev = check_device();
    if (dev != VQ_OK)
        return dev;
    return status(vq::launch_row_quant(x, x_dtype, q_out, scales_out, (int)n_rows, (int)k,
                                       static_cast<hipStream_t>(stream)));
}

int vq_rotate(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int dtype, const float *inv_freq,
              const int32_t *ctx_len, const uint64_t *tree_mask, void *q_out, int64_t q_out_stride, void *k_out,
              int64_t k_out_stride, int64_t batch, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
              int64_t rot_dim, int interleaved, float scale, void *stream) {
    if (!q || !q_out || !inv_freq || !ctx_len || (!k) != (!k_out))
        return VQ_ERR_NULL_POINTER;
    if (!half_type(dtype))
        return VQ_ERR_BAD_DTYPE;
    const auto stride_ok = [](int64_t s, int64_t width) { return s % 8 == 0 && in(s, width, VQ_MAX_DIM); };
    if (!in(batch, 1, VQ_MAX_DIM) || !in(n, 1, tree_mask ? VQ_MAX_TREE_NODES : VQ_MAX_DIM) ||
        batch * n > VQ_MAX_DIM / 2 || !in(q_heads, 1, VQ_MAX_HEADS) || (k && !in(kv_heads, 1, VQ_MAX_HEADS)) ||
        !in(head_dim, 16, VQ_MAX_ROTATE_DIM) || head_dim % 16 || !in(rot_dim, 16, head_dim) || rot_dim % 16 ||
        !stride_ok(q_stride, q_heads * head_dim) || !stride_ok(q_out_stride, q_heads * head_dim) ||
        (k && (!stride_ok(k_stride, kv_heads * head_dim) || !stride_ok(k_out_stride, kv_heads * head_dim))))
        return VQ_ERR_BAD_SHAPE;
    if (!aligned({q, k, q_out, k_out}, 16) || !aligned({tree_mask}, 8) || !aligned({inv_freq, ctx_len}, 4))
        return VQ_ERR_MISALIGNED;
    const int dev = check_device();
    if (dev != VQ_OK)
        return dev;
    return status(vq::launch_rotate({q, q_stride, k, k_stride, dtype, inv_freq, ctx_len, tree_mask, q_out,
                                     q_out_stride, k_out, k_out_stride, (int)batch, (int)n, (int)q_heads,
                                     (int)kv_heads, (int)head_dim, (int)rot_dim, interleaved != 0, scale,
                                     static_cast<hipStream_t>(stream)}));
}

}  // extern "C"
