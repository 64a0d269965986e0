// layer_internal.h -- host-side declarations of the decoder-layer operators
// (8-bit products, residual norm, row quantization, rotation).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "vq.h"

namespace vq {

// Arguments of one 8-bit product, already checked.  `up` null: out[n][m] of
// one matrix; else the gated form: `w` holds the gate's rows, `up` the other
// factor's, and out[n][m] = act(gate) * up.
struct W8A8Args {
    const int8_t *w, *up;
    const float *w_scales, *up_scales;
    const int8_t *x;
    const float *x_scales;
    const float *bias;  // or null; plain form only
    int activation;
    void *out;
    int out_dtype;
    int N, M, K;
    void *workspace;  // or null
    size_t workspace_bytes;
    hipStream_t stream;
};
hipError_t launch_w8a8(const W8A8Args &a);
size_t w8a8_workspace(int N);  // for N rows of any product
size_t w8a8_workspace_used(int N, int M, int K, bool gated);  // of that

// Arguments of one residual update with its norms, already checked.
struct RowNormArgs {
    const void *residual;
    int residual_dtype;
    const void *y;  // or null
    int y_dtype;
    const float *post_weight;
    const void *gate;
    bool gate_rows;  // gate [n][c] of y's type, else fp32 [c]
    float alpha;
    const float *weight;
    float eps;
    void *residual_out;  // or null
    void *out;
    int out_dtype;  // I8: with scales_out
    float *scales_out;
    int N, C;
    hipStream_t stream;
};
hipError_t launch_row_norm(const RowNormArgs &a);
hipError_t launch_row_quant(const void *x, int x_dtype, int8_t *q, float *scales, int N, int C, hipStream_t stream);

// Arguments of one rotation, already checked.
struct RotateArgs {
    const void *q;
    int64_t q_stride;
    const void *k;  // or null
    int64_t k_stride;
    int dtype;
    const float *inv_freq;
    const int32_t *ctx_len;
    const uint64_t *tree_mask;  // or null: a chain
    void *q_out;
    int64_t q_out_stride;
    void *k_out;
    int64_t k_out_stride;
    int batch, n, q_heads, kv_heads, head_dim, rot_dim;
    bool interleaved;
    float scale;
    hipStream_t stream;
};
hipError_t launch_rotate(const RotateArgs &a);

}  // namespace vq
