// Internal interface between the host entry points of the layer operators
// (ssu_layer_api.cpp) and their gfx950 kernels (ssu_norm.hip, ssu_mx.hip,
// ssu_logprob.hip).
#pragma once

#include <stdint.h>

#include "../../include/ssu.h"

namespace ssu {

// What the launch functions return, besides HIP's codes: more work items than the 2^32 - 1 of one launch.
constexpr int kTooManyWorkItems = -1;

// RMS norm. Strides are in elements; a "part" is one group of one row.
struct NormParams {
    const void *x, *weight, *residual, *gate;  // residual, gate may be null
    void *out, *residual_out;
    uint8_t *scales;  // MX outputs
    int64_t x_s, res_s, gate_s, out_s, res_out_s;
    int64_t parts;  // rows * groups
    int32_t groups, part;  // groups per row, elements per part
    int32_t weight_f32, res_f32;
    float eps;
};
int launch_norm(const NormParams &p, int dtype, int format, void *stream);

// Rows to MXFP8 / MXFP4: `blocks` = k / 32 per row; codes and scales contiguous.
int launch_mx_quantize_rows(const void *src, int dtype, int64_t stride, int64_t rows, int64_t k, uint8_t *codes,
                            uint8_t *scales, int format, void *stream);

// Product with MXFP4 weights. Strides: codes and scales in bytes, out in
// elements. Up to kMxRowsMax rows run in the streaming kernel, which reads
// scales where they are (and quantises up to kMxFuseRows rows by itself); more rows run
// in the tiled kernels, whose quantised codes and laid out scales are in a workspace.
constexpr int kMxRowsMax = 16;
constexpr int kMxFuseRows = 4;
struct MxParams {
    const void *x;  // float activations, or null
    const uint8_t *a, *a_scale, *w, *w_scale;
    const void *bias;  // may be null
    void *out;
    int64_t x_s, a_s, as_s, w_s, ws_s, out_s;
    int32_t m, n, k;
    int32_t bias_f32;
    int32_t x_dtype;
    uint8_t *workspace;
};
// Workspace bytes of a product whose activations come as floats or as codes.
int64_t mx_linear_workspace(int64_t m, int64_t n, int64_t k, int format, bool floats);
int launch_mx_linear(const MxParams &p, int format, int out_dtype, void *stream);

// Token log probabilities. Strides in elements.
struct LogprobParams {
    const void *logits, *tokens;
    const int32_t *mask;       // may be null
    const float *temperature;  // may be null
    float *logprob, *entropy, *top_logprobs;
    int32_t *rank, *top_tokens;
    int64_t logits_s, tokens_s, mask_s, temp_s;
    int64_t rows;
    int32_t vocab, top, tokens_i64;
    uint8_t *workspace;
};
// Workspace bytes (0 where a row is not split).
int64_t logprobs_workspace(int64_t rows, int64_t vocab, int64_t top);
int launch_logprobs(const LogprobParams &p, int dtype, void *stream);

}  // namespace ssu
