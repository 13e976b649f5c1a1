// Internal interface between the host entry points of the layer operators
// (ssu_layer_api.cpp) and their gfx950 kernels (ssu_norm.hip, ssu_mx.hip,
// ssu_logprob.hip, ssu_lora.hip, ssu_beam.hip, ssu_reorder.hip).
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

// Low-rank adapters. Strides in elements (x's and its scales' in bytes for codes).
struct LoraParams {
    const void *x, *a, *b, *ids;
    const uint8_t *x_scale;  // of codes
    const float *scale;      // may be null
    void *y;
    int64_t x_s, xs_s, a_l, a_r, b_l, b_n, ids_s, scale_s, y_s;
    int32_t rows, k, n, rank, adapters, ids_i64;
    int32_t slices, slice;  // of k; set by the launch, like the rows of a tile of the second product
    int32_t up_rows, parts;
    uint8_t *workspace;
};
int64_t lora_workspace(int64_t rows, int64_t adapters, int64_t k, int64_t n, int64_t rank);
int launch_add_lora(const LoraParams &p, int dtype, int format, void *stream);

// Beam search: choice of continuations. Strides in elements.
struct BeamParams {
    const void *logits;
    const float *scores;
    const uint8_t *finished;  // may be null
    const int32_t *mask;      // may be null
    float *out_scores;
    int32_t *out_parents, *out_tokens;
    int64_t logits_s, scores_b, scores_s, finished_b, finished_s, mask_s;
    int64_t batch;
    int32_t beams, vocab, keep, end_token;
    uint8_t *workspace;
};
int64_t beam_workspace(int64_t rows, int64_t beams, int64_t vocab, int64_t keep, int dtype);
int launch_beam_select(const BeamParams &p, int dtype, void *stream);

// Beam search: states after the choice. Strides of slots, parents and out in elements, of a
// pool in bytes.
constexpr int kReorderPools = 64;  // of one launch
struct ReorderPool {
    uint8_t *base;
    int64_t stride, bytes;  // of a slot
    int64_t slots;
};
struct ReorderParams {
    const void *slots, *parents;
    void *out;
    int64_t slots_b, slots_s, parents_b, parents_s, out_b;
    int64_t batch, piece;  // bytes of a slot that a workgroup copies; set by plan_reorder
    int32_t beams, count;
    int32_t slots_i64, parents_i64, out_i64;
    int32_t first_piece[kReorderPools + 1];  // set by plan_reorder
    ReorderPool pool[kReorderPools];
};
int plan_reorder(ReorderParams &p);  // 0, or kTooManyWorkItems
int launch_reorder(const ReorderParams &p, void *stream);

}  // namespace ssu
