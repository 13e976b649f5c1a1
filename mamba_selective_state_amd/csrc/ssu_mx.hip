// Rows to MXFP8 / MXFP4 (ssu_mx_quantize) and the product of such rows with
// MXFP4 weights (ssu_mx_linear) on the block-scaled matrix instructions.
#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kQuantThreads = 256;

// Four lanes per block of 32 values, eight each.
template <typename T, int FORMAT>
__global__ __launch_bounds__(kQuantThreads) void mx_quantize_rows_kernel(const T *src, int64_t stride, int64_t rows,
                                                                         int32_t k, uint8_t *codes, uint8_t *scales) {
    const int64_t eighths = k / 8;  // per row
    const int64_t total = rows * eighths;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQuantThreads;
    // four lanes of a block are live or not together: a row is a multiple of four eighths
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x; i < total; i += step) {
        const int64_t row = i / eighths, at = (i % eighths) * 8;
        float v[8];
        load8(src + row * stride + at, v);
        uint32_t code[2];
        const uint32_t s = mx_block<FORMAT>(v, code);
        store_codes<FORMAT>(codes + row * (FORMAT == SSU_FORMAT_MXFP4 ? k / 2 : k), at, code);
        if (i % 4 == 0)
            scales[i / 4] = static_cast<uint8_t>(s);
    }
}

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// One wave per 32 x 32 tile of the output; both operands straight from
// memory. Operands of the 32x32x64 instruction (checked on the device): lane l
// is row l % 32; E2M1 codes k = 32 (l / 32) + 0..31 in the first four
// registers; E4M3 codes k = 16 (l / 32) + 0..15 in the first four and k = 32 +
// 16 (l / 32) + 0..15 in the last; the scale byte of block l / 32.
// Result: register i is row i % 4 + 8 (i / 4) + 4 (l / 32), column l % 32.
template <typename OT, int FORMAT>
__global__ __launch_bounds__(64) void mx_linear_kernel(const MxParams p) {
    const int l = threadIdx.x, r = l % 32, h = l / 32;
    const int m0 = static_cast<int>(blockIdx.y) * 32, n0 = static_cast<int>(blockIdx.x) * 32;
    // rows past the end read the last row; their results are not stored
    const int ra = min(m0 + r, p.m - 1), rb = min(n0 + r, p.n - 1);
    const uint8_t *a = p.a + ra * p.a_s, *w = p.w + rb * p.w_s;
    const uint8_t *as = p.a_scale + ra * p.as_s, *ws = p.w_scale + rb * p.ws_s;
    f32x16 acc = {};
    const int blocks = p.k / 32;
    for (int b = 0; b < blocks; b += 2) {
        const bool both = b + 1 < blocks;
        const bool live = h == 0 || both;
        i32x8 av = {}, wv = {};
        if constexpr (FORMAT == SSU_FORMAT_MXFP8) {
            const i32x4 lo = *reinterpret_cast<const i32x4 *>(a + b * 32 + 16 * h);
            i32x4 hi = {};
            if (both)
                hi = *reinterpret_cast<const i32x4 *>(a + b * 32 + 32 + 16 * h);
            av = i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        } else if (live) {
            const i32x4 v = *reinterpret_cast<const i32x4 *>(a + (b + h) * 16);
            av = i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
        }
        int sa = 127, sw = 127;
        if (live) {
            const i32x4 v = *reinterpret_cast<const i32x4 *>(w + (b + h) * 16);
            wv = i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
            sa = as[b + h];
            sw = ws[b + h];
        }
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, wv, acc, FORMAT == SSU_FORMAT_MXFP8 ? 0 : 4, 4, 0,
                                                              sa, 0, sw);
    }
    const int n = n0 + r;
    if (n >= p.n)
        return;
    float bias = 0.0f;
    if (p.bias)
        bias = p.bias_f32 ? static_cast<const float *>(p.bias)[n] : widen(static_cast<const OT *>(p.bias)[n]);
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int m = m0 + i % 4 + 8 * (i / 4) + 4 * h;
        if (m < p.m)
            static_cast<OT *>(p.out)[m * p.out_s + n] = narrow<OT>(acc[i] + bias);
    }
}

template <typename T>
const void *quantize_fn(int format) {
    return format == SSU_FORMAT_MXFP4 ? reinterpret_cast<const void *>(&mx_quantize_rows_kernel<T, SSU_FORMAT_MXFP4>)
                                      : reinterpret_cast<const void *>(&mx_quantize_rows_kernel<T, SSU_FORMAT_MXFP8>);
}
template <typename OT>
const void *linear_fn(int format) {
    return format == SSU_FORMAT_MXFP4 ? reinterpret_cast<const void *>(&mx_linear_kernel<OT, SSU_FORMAT_MXFP4>)
                                      : reinterpret_cast<const void *>(&mx_linear_kernel<OT, SSU_FORMAT_MXFP8>);
}

}  // namespace

int launch_mx_quantize_rows(const void *src, int dtype, int64_t stride, int64_t rows, int64_t k, uint8_t *codes,
                            uint8_t *scales, int format, void *stream) {
    const void *fn = dtype == SSU_F32   ? quantize_fn<float>(format)
                     : dtype == SSU_F16 ? quantize_fn<_Float16>(format)
                                        : quantize_fn<__bf16>(format);
    int64_t blocks = (rows * (k / 8) + kQuantThreads - 1) / kQuantThreads;
    blocks = blocks > 65536 ? 65536 : blocks;
    int32_t k32 = static_cast<int32_t>(k);
    void *args[] = {&src, &stride, &rows, &k32, &codes, &scales};
    return static_cast<int>(hipLaunchKernel(fn, dim3(static_cast<unsigned>(blocks)), dim3(kQuantThreads), args, 0,
                                            static_cast<hipStream_t>(stream)));
}

int launch_mx_linear(const MxParams &p, int format, int out_dtype, void *stream) {
    const void *fn = out_dtype == SSU_F32   ? linear_fn<float>(format)
                     : out_dtype == SSU_F16 ? linear_fn<_Float16>(format)
                                            : linear_fn<__bf16>(format);
    MxParams pc = p;
    void *args[] = {&pc};
    // grid.y ends at 65535
    if ((p.m + 31) / 32 > 65535)
        return static_cast<int>(hipErrorInvalidValue);
    return static_cast<int>(hipLaunchKernel(fn, dim3((p.n + 31) / 32, (p.m + 31) / 32), dim3(64), args, 0,
                                            static_cast<hipStream_t>(stream)));
}

}  // namespace ssu
