// Host entry points of the layer operators (norm, MX product, token log
// probabilities): argument validation and launches, with the conventions of
// ssu_api.cpp -- only shapes, strides, dtypes and alignment are looked at.
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/ssu.h"
#include "ssu_internal.h"
#include "ssu_layer.h"

namespace {

ssu_status_t fail(ssu_status_t st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return ssu::report_error(st, buf);
}

ssu_status_t done(int hip) {
    if (hip == ssu::kTooManyWorkItems)
        return fail(SSU_ERR_NOT_IMPLEMENTED, "more rows or outputs than one launch takes");
    if (hip != 0)
        return fail(SSU_ERR_HIP, "kernel launch failed: %s", ssu::hip_error_string(hip));
    return ssu::report_error(SSU_OK, "");
}

// Rows, columns and inner sizes. The kernels count in 32 bits within a row and round sizes up to
// whole accesses, tiles and rounds of tiles, a few KiB at most.
constexpr int64_t kMostSize = INT32_MAX - 65536;

bool is_float(int d) { return d == SSU_F32 || d == SSU_F16 || d == SSU_BF16; }
bool is_index(int d) { return d == SSU_I32 || d == SSU_I64; }
int64_t elem_bytes(int d) { return d == SSU_F32 || d == SSU_I32 ? 4 : d == SSU_U8 ? 1 : d == SSU_I64 ? 8 : 2; }
bool present(const ssu_tensor_t &t) { return t.data != nullptr; }
bool aligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

// A [rows, cols] tensor whose rows are contiguous; an output's rows must not
// overlap. Its row stride goes to `stride`.
ssu_status_t matrix(const char *name, const ssu_tensor_t &t, int64_t rows, int64_t cols, bool output, int64_t *stride) {
    if (!present(t))
        return fail(SSU_ERR_VALUE, "%s is required", name);
    if (t.ndim != 2 || t.size[0] != rows || t.size[1] != cols)
        return fail(SSU_ERR_VALUE, "%s must be [%lld, %lld]", name, (long long)rows, (long long)cols);
    if (cols > 1 && t.stride[1] != 1)
        return fail(SSU_ERR_VALUE, "%s needs last stride 1", name);
    if (rows > 1 && t.stride[0] < (output ? cols : 0))
        return fail(SSU_ERR_VALUE, output ? "%s has overlapping rows" : "%s has a negative stride", name);
    if (!aligned(t.data, elem_bytes(t.dtype)))
        return fail(SSU_ERR_VALUE, "%s is not aligned to its element size", name);
    *stride = rows > 1 && cols > 0 ? t.stride[0] : cols;
    return SSU_OK;
}

ssu_status_t vector(const char *name, const ssu_tensor_t &t, int64_t n, bool contiguous, int64_t *stride) {
    if (!present(t))
        return fail(SSU_ERR_VALUE, "%s is required", name);
    if (t.ndim != 1 || t.size[0] != n)
        return fail(SSU_ERR_VALUE, "%s must be [%lld]", name, (long long)n);
    if (n > 1 && (contiguous ? t.stride[0] != 1 : t.stride[0] < 0))
        return fail(SSU_ERR_VALUE, contiguous ? "%s needs stride 1" : "%s has a negative stride", name);
    if (!aligned(t.data, elem_bytes(t.dtype)))
        return fail(SSU_ERR_VALUE, "%s is not aligned to its element size", name);
    if (stride)
        *stride = n > 1 ? t.stride[0] : 0;
    return SSU_OK;
}

// Contiguous MX codes and scales of [rows, k].
ssu_status_t mx_output(const ssu_tensor_t &codes, const ssu_tensor_t &scales, const char *codes_name,
                       const char *scales_name, int64_t rows, int64_t k, int format) {
    int64_t s;
    if (!present(scales))
        return fail(SSU_ERR_VALUE, "%s is required", scales_name);
    if (codes.dtype != SSU_U8 || scales.dtype != SSU_U8)
        return fail(SSU_ERR_VALUE, "%s and %s must be u8", codes_name, scales_name);
    const int64_t cols = format == SSU_FORMAT_MXFP4 ? k / 2 : k;
    if (ssu_status_t st = matrix(codes_name, codes, rows, cols, true, &s))
        return st;
    if (s != cols)
        return fail(SSU_ERR_VALUE, "%s must be contiguous", codes_name);
    if (ssu_status_t st = matrix(scales_name, scales, rows, k / 32, true, &s))
        return st;
    if (s != k / 32)
        return fail(SSU_ERR_VALUE, "%s must be contiguous", scales_name);
    if (!aligned(codes.data, 8))
        return fail(SSU_ERR_VALUE, "%s must be 8-byte aligned", codes_name);
    return SSU_OK;
}

bool mx_format(int f) { return f == SSU_FORMAT_MXFP4 || f == SSU_FORMAT_MXFP8; }

// MX operand of the product: codes of `cols` bytes a row and k / 32 scales.
ssu_status_t mx_operand(const char *name, const ssu_tensor_t &codes, const ssu_tensor_t &scales, int64_t rows,
                        int64_t cols, int64_t k, int64_t *codes_s, int64_t *scales_s) {
    char scale_name[32];
    snprintf(scale_name, sizeof scale_name, "%s_scale", name);
    if (codes.dtype != SSU_U8)
        return fail(SSU_ERR_VALUE, "%s must be u8 codes", name);
    if (ssu_status_t st = matrix(name, codes, rows, cols, false, codes_s))
        return st;
    if (!present(scales) || scales.dtype != SSU_U8)
        return fail(SSU_ERR_VALUE, "%s must be given, as u8", scale_name);
    if (ssu_status_t st = matrix(scale_name, scales, rows, k / 32, false, scales_s))
        return st;
    if (!aligned(codes.data, 16) || *codes_s % 16 != 0)
        return fail(SSU_ERR_VALUE, "%s needs a 16-byte aligned base and row stride", name);
    return SSU_OK;
}

}  // namespace

extern "C" {

ssu_status_t ssu_add_rms_norm(const ssu_norm_args_t *a, void *stream) {
    if (!a)
        return fail(SSU_ERR_VALUE, "ssu_add_rms_norm: args is NULL");
    const ssu_tensor_t &x = a->x;
    if (!present(x) || x.ndim != 2)
        return fail(SSU_ERR_VALUE, "x must be [rows, dim]");
    if (!is_float(x.dtype))
        return fail(SSU_ERR_VALUE, "x must be f32, f16 or bf16");
    const int64_t rows = x.size[0], dim = x.size[1];
    if (rows < 0 || dim < 0 || dim > kMostSize)
        return fail(SSU_ERR_VALUE, "x has a size out of range");
    ssu::NormParams p = {};
    if (ssu_status_t st = matrix("x", x, rows, dim, false, &p.x_s))
        return st;
    if (a->groups < 1 || dim % a->groups != 0)
        return fail(SSU_ERR_VALUE, "groups must divide dim");
    if (!(a->eps >= 0.0f) || isinf(a->eps))
        return fail(SSU_ERR_VALUE, "eps must be finite and not negative");
    if (ssu_status_t st = vector("weight", a->weight, dim, true, nullptr))
        return st;
    if (a->weight.dtype != x.dtype && a->weight.dtype != SSU_F32)
        return fail(SSU_ERR_VALUE, "weight must have x's dtype or be f32");
    if (present(a->gate)) {
        if (a->gate.dtype != x.dtype)
            return fail(SSU_ERR_VALUE, "gate must have x's dtype");
        if (ssu_status_t st = matrix("gate", a->gate, rows, dim, false, &p.gate_s))
            return st;
    }
    if (present(a->residual) != present(a->residual_out))
        return fail(SSU_ERR_VALUE, "residual and residual_out go together");
    if (present(a->residual)) {
        if (a->residual.dtype != a->residual_out.dtype || (a->residual.dtype != x.dtype && a->residual.dtype != SSU_F32))
            return fail(SSU_ERR_VALUE, "residual and residual_out must both have x's dtype or both be f32");
        if (ssu_status_t st = matrix("residual", a->residual, rows, dim, false, &p.res_s))
            return st;
        if (ssu_status_t st = matrix("residual_out", a->residual_out, rows, dim, true, &p.res_out_s))
            return st;
    }
    if (!present(a->out))
        return fail(SSU_ERR_VALUE, "out is required");
    if (a->out_format == SSU_FORMAT_SAME) {
        if (a->out.dtype != x.dtype)
            return fail(SSU_ERR_VALUE, "out must have x's dtype");
        if (present(a->out_scales))
            return fail(SSU_ERR_VALUE, "out_scales belongs to the MX formats");
        if (ssu_status_t st = matrix("out", a->out, rows, dim, true, &p.out_s))
            return st;
    } else if (mx_format(a->out_format)) {
        if ((dim / a->groups) % 32 != 0)
            return fail(SSU_ERR_VALUE, "an MX output needs dim / groups to be a multiple of 32");
        if (ssu_status_t st = mx_output(a->out, a->out_scales, "out", "out_scales", rows, dim, a->out_format))
            return st;
        p.out_s = a->out_format == SSU_FORMAT_MXFP4 ? dim / 2 : dim;
    } else {
        return fail(SSU_ERR_NOT_IMPLEMENTED, "out_format must be SAME, MXFP8 or MXFP4");
    }
    if (rows == 0 || dim == 0)
        return done(0);
    p.x = x.data;
    p.weight = a->weight.data;
    p.residual = a->residual.data;
    p.gate = a->gate.data;
    p.out = const_cast<void *>(a->out.data);
    p.residual_out = const_cast<void *>(a->residual_out.data);
    p.scales = static_cast<uint8_t *>(const_cast<void *>(a->out_scales.data));
    p.groups = static_cast<int32_t>(a->groups);
    p.part = static_cast<int32_t>(dim / a->groups);
    p.parts = rows * a->groups;
    if (rows > INT32_MAX / a->groups)
        return fail(SSU_ERR_NOT_IMPLEMENTED, "rows * groups too large");
    p.weight_f32 = a->weight.dtype == SSU_F32;
    p.res_f32 = present(a->residual) && a->residual.dtype == SSU_F32;
    p.eps = a->eps;
    return done(ssu::launch_norm(p, x.dtype, a->out_format, stream));
}

ssu_status_t ssu_mx_quantize(const ssu_tensor_t *src, const ssu_tensor_t *codes, const ssu_tensor_t *scales,
                             int32_t format, void *stream) {
    if (!src || !codes || !scales)
        return fail(SSU_ERR_VALUE, "ssu_mx_quantize: a tensor is NULL");
    if (!mx_format(format))
        return fail(SSU_ERR_NOT_IMPLEMENTED, "format must be MXFP8 or MXFP4");
    if (!present(*src) || src->ndim != 2 || !is_float(src->dtype))
        return fail(SSU_ERR_VALUE, "src must be [rows, k], f32, f16 or bf16");
    const int64_t rows = src->size[0], k = src->size[1];
    if (k % 32 != 0)
        return fail(SSU_ERR_VALUE, "k must be a multiple of 32");
    if (k > kMostSize)
        return fail(SSU_ERR_NOT_IMPLEMENTED, "k too large");
    int64_t s;
    if (ssu_status_t st = matrix("src", *src, rows, k, false, &s))
        return st;
    if (ssu_status_t st = mx_output(*codes, *scales, "codes", "scales", rows, k, format))
        return st;
    if (rows == 0 || k == 0)
        return done(0);
    return done(ssu::launch_mx_quantize_rows(src->data, src->dtype, s, rows, k,
                                             static_cast<uint8_t *>(const_cast<void *>(codes->data)),
                                             static_cast<uint8_t *>(const_cast<void *>(scales->data)), format, stream));
}

int64_t ssu_mx_linear_workspace_bytes(const ssu_mx_linear_args_t *a) {
    if (!a || a->x.ndim != 2 || a->w.ndim != 2 || !mx_format(a->x_format))
        return 0;
    return ssu::mx_linear_workspace(a->x.size[0], a->w.size[0], a->w.size[1] * 2, a->x_format, is_float(a->x.dtype));
}

ssu_status_t ssu_mx_linear(const ssu_mx_linear_args_t *a, void *workspace, int64_t workspace_bytes, void *stream) {
    if (!a)
        return fail(SSU_ERR_VALUE, "ssu_mx_linear: args is NULL");
    if (!mx_format(a->x_format))
        return fail(SSU_ERR_NOT_IMPLEMENTED, "x_format must be MXFP8 or MXFP4");
    if (!present(a->x) || a->x.ndim != 2 || !present(a->w) || a->w.ndim != 2 || !present(a->out) || a->out.ndim != 2)
        return fail(SSU_ERR_VALUE, "x, w and out must be 2-D");
    const int64_t m = a->x.size[0], n = a->w.size[0], k = a->w.size[1] * 2;
    if (m < 0 || n < 0 || m > kMostSize || n > kMostSize || k > kMostSize)
        return fail(SSU_ERR_VALUE, "x or w has a size out of range");
    if (k % 32 != 0)
        return fail(SSU_ERR_VALUE, "k must be a multiple of 32 (w is [n, k / 2] code pairs)");
    ssu::MxParams p = {};
    if (ssu_status_t st = mx_operand("w", a->w, a->w_scale, n, k / 2, k, &p.w_s, &p.ws_s))
        return st;
    const bool floats = is_float(a->x.dtype);
    if (floats) {
        if (present(a->x_scale))
            return fail(SSU_ERR_VALUE, "x_scale belongs to u8 codes");
        if (ssu_status_t st = matrix("x", a->x, m, k, false, &p.x_s))
            return st;
    } else if (ssu_status_t st = mx_operand("x", a->x, a->x_scale, m, a->x_format == SSU_FORMAT_MXFP4 ? k / 2 : k, k,
                                            &p.a_s, &p.as_s)) {
        return st;
    }
    if (!is_float(a->out.dtype))
        return fail(SSU_ERR_VALUE, "out must be f32, f16 or bf16");
    if (ssu_status_t st = matrix("out", a->out, m, n, true, &p.out_s))
        return st;
    if (present(a->bias)) {
        if (a->bias.dtype != SSU_F32 && a->bias.dtype != a->out.dtype)
            return fail(SSU_ERR_VALUE, "bias must be f32 or have out's dtype");
        if (ssu_status_t st = vector("bias", a->bias, n, true, nullptr))
            return st;
    }
    if (m == 0 || n == 0)
        return done(0);
    const int64_t need = ssu_mx_linear_workspace_bytes(a);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(SSU_ERR_VALUE, "workspace must be 256-byte aligned and hold %lld bytes", (long long)need);
    p.workspace = static_cast<uint8_t *>(workspace);
    if (floats) {
        p.x = a->x.data;
        p.x_dtype = a->x.dtype;
    } else {
        p.a = static_cast<const uint8_t *>(a->x.data);
        p.a_scale = static_cast<const uint8_t *>(a->x_scale.data);
    }
    p.w = static_cast<const uint8_t *>(a->w.data);
    p.w_scale = static_cast<const uint8_t *>(a->w_scale.data);
    p.bias = a->bias.data;
    p.bias_f32 = present(a->bias) && a->bias.dtype == SSU_F32;
    p.out = const_cast<void *>(a->out.data);
    p.m = static_cast<int32_t>(m);
    p.n = static_cast<int32_t>(n);
    p.k = static_cast<int32_t>(k);
    return done(ssu::launch_mx_linear(p, a->x_format, a->out.dtype, stream));
}

int64_t ssu_token_logprobs_workspace_bytes(const ssu_logprob_args_t *a) {
    if (!a || a->logits.ndim != 2 || a->logits.size[0] <= 0)
        return 0;
    return ssu::logprobs_workspace(a->logits.size[0], a->logits.size[1], present(a->top_tokens) ? a->top_tokens.size[1] : 0);
}

ssu_status_t ssu_token_logprobs(const ssu_logprob_args_t *a, void *workspace, int64_t workspace_bytes, void *stream) {
    if (!a)
        return fail(SSU_ERR_VALUE, "ssu_token_logprobs: args is NULL");
    const ssu_tensor_t &x = a->logits;
    if (!present(x) || x.ndim != 2 || !is_float(x.dtype))
        return fail(SSU_ERR_VALUE, "logits must be [rows, vocab], f32, f16 or bf16");
    const int64_t rows = x.size[0], vocab = x.size[1];
    if (rows < 0 || vocab < 0 || rows > INT32_MAX || vocab > kMostSize)
        return fail(SSU_ERR_VALUE, "logits has a size out of range");
    ssu::LogprobParams p = {};
    if (ssu_status_t st = matrix("logits", x, rows, vocab, false, &p.logits_s))
        return st;
    if (!is_index(a->tokens.dtype))
        return fail(SSU_ERR_VALUE, "tokens must be i32 or i64");
    if (ssu_status_t st = vector("tokens", a->tokens, rows, false, &p.tokens_s))
        return st;
    if (present(a->mask)) {
        if (a->mask.dtype != SSU_I32)
            return fail(SSU_ERR_VALUE, "mask must be i32 words of 32 bits");
        if (ssu_status_t st = matrix("mask", a->mask, rows, (vocab + 31) / 32, false, &p.mask_s))
            return st;
    }
    if (present(a->temperature)) {
        if (a->temperature.dtype != SSU_F32)
            return fail(SSU_ERR_VALUE, "temperature must be f32");
        if (ssu_status_t st = vector("temperature", a->temperature, rows, false, &p.temp_s))
            return st;
    }
    if (a->logprob.dtype != SSU_F32 || a->entropy.dtype != SSU_F32 || a->rank.dtype != SSU_I32)
        return fail(SSU_ERR_VALUE, "logprob and entropy must be f32, rank i32");
    if (ssu_status_t st = vector("logprob", a->logprob, rows, true, nullptr))
        return st;
    if (ssu_status_t st = vector("entropy", a->entropy, rows, true, nullptr))
        return st;
    if (ssu_status_t st = vector("rank", a->rank, rows, true, nullptr))
        return st;
    if (present(a->top_tokens) != present(a->top_logprobs))
        return fail(SSU_ERR_VALUE, "top_tokens and top_logprobs go together");
    int64_t top = 0;
    if (present(a->top_tokens)) {
        if (a->top_tokens.ndim != 2 || a->top_tokens.dtype != SSU_I32 || a->top_logprobs.dtype != SSU_F32)
            return fail(SSU_ERR_VALUE, "top_tokens must be i32 and top_logprobs f32, [rows, top]");
        top = a->top_tokens.size[1];
        if (top < 0 || top > SSU_TOP_MAX)
            return fail(SSU_ERR_NOT_IMPLEMENTED, "top must be at most %d", SSU_TOP_MAX);
        int64_t s;
        if (ssu_status_t st = matrix("top_tokens", a->top_tokens, rows, top, true, &s))
            return st;
        if (s != top)
            return fail(SSU_ERR_VALUE, "top_tokens must be contiguous");
        if (ssu_status_t st = matrix("top_logprobs", a->top_logprobs, rows, top, true, &s))
            return st;
        if (s != top)
            return fail(SSU_ERR_VALUE, "top_logprobs must be contiguous");
    }
    if (rows == 0)
        return done(0);
    p.logits = x.data;
    p.tokens = a->tokens.data;
    p.tokens_i64 = a->tokens.dtype == SSU_I64;
    p.mask = static_cast<const int32_t *>(a->mask.data);
    p.temperature = static_cast<const float *>(a->temperature.data);
    p.logprob = static_cast<float *>(const_cast<void *>(a->logprob.data));
    p.entropy = static_cast<float *>(const_cast<void *>(a->entropy.data));
    p.rank = static_cast<int32_t *>(const_cast<void *>(a->rank.data));
    p.top_tokens = static_cast<int32_t *>(const_cast<void *>(a->top_tokens.data));
    p.top_logprobs = static_cast<float *>(const_cast<void *>(a->top_logprobs.data));
    p.rows = rows;
    p.vocab = static_cast<int32_t>(vocab);
    p.top = static_cast<int32_t>(top);
    const int64_t need = ssu::logprobs_workspace(rows, vocab, top);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(SSU_ERR_VALUE, "workspace must be 256-byte aligned and hold %lld bytes", (long long)need);
    p.workspace = static_cast<uint8_t *>(workspace);
    return done(ssu::launch_logprobs(p, x.dtype, stream));
}

}  // extern "C"
