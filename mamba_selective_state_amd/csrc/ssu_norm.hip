// Gated, residual-adding RMS norm (ssu_add_rms_norm): per part of a row,
//   u = x * silu(gate) + residual,  y = u * rsqrt(mean u^2 + eps) * weight.
#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kNormThreads = 256;

// Eight values of u at `at` of row `row` (n of them exist).
template <typename T>
__device__ __forceinline__ void load_u(const NormParams &p, int64_t row, int at, int n, float u[8]) {
    load8(static_cast<const T *>(p.x) + row * p.x_s + at, n, u);
    if (p.gate) {
        float z[8];
        load8(static_cast<const T *>(p.gate) + row * p.gate_s + at, n, z);
#pragma unroll
        for (int i = 0; i < 8; i++)
            u[i] *= z[i] / (1.0f + __expf(-z[i]));
    }
    if (p.residual) {
        float r[8];
        if (p.res_f32)
            load8(static_cast<const float *>(p.residual) + row * p.res_s + at, n, r);
        else
            load8(static_cast<const T *>(p.residual) + row * p.res_s + at, n, r);
#pragma unroll
        for (int i = 0; i < 8; i++)
            u[i] += r[i];
    }
}

template <typename T, int FORMAT>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(const NormParams p) {
    __shared__ float sums[kNormThreads / kWaveLanes];
    const int64_t part = blockIdx.x;
    const int64_t row = part / p.groups;
    const int first = static_cast<int>(part % p.groups) * p.part;
    const int tid = threadIdx.x;
    float ss = 0.0f;
    for (int i = tid * 8; i < p.part; i += kNormThreads * 8) {
        float u[8];
        load_u<T>(p, row, first + i, min(8, p.part - i), u);
#pragma unroll
        for (int j = 0; j < 8; j++)
            ss += u[j] * u[j];
    }
#pragma unroll
    for (int d = 1; d < kWaveLanes; d *= 2)
        ss += __shfl_xor(ss, d);
    if (tid % kWaveLanes == 0)
        sums[tid / kWaveLanes] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < kNormThreads / kWaveLanes; w++)
        ss += sums[w];
    const float scale = 1.0f / sqrtf(ss / static_cast<float>(p.part) + p.eps);
    for (int i = tid * 8; i < p.part; i += kNormThreads * 8) {
        const int n = min(8, p.part - i);
        float u[8], g[8];
        load_u<T>(p, row, first + i, n, u);
        if (p.weight_f32)
            load8(static_cast<const float *>(p.weight) + first + i, n, g);
        else
            load8(static_cast<const T *>(p.weight) + first + i, n, g);
        if (p.residual) {
            if (p.res_f32)
                store8(static_cast<float *>(p.residual_out) + row * p.res_out_s + first + i, n, u);
            else
                store8(static_cast<T *>(p.residual_out) + row * p.res_out_s + first + i, n, u);
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
            u[j] = u[j] * scale * g[j];
        if constexpr (FORMAT == SSU_FORMAT_SAME) {
            store8(static_cast<T *>(p.out) + row * p.out_s + first + i, n, u);
        } else {
            uint32_t code[2];
            const uint32_t s = mx_block<FORMAT>(u, code);
            store_codes<FORMAT>(static_cast<uint8_t *>(p.out) + row * p.out_s, first + i, code);
            if (tid % 4 == 0)
                p.scales[(row * p.groups * p.part + first + i) / 32] = static_cast<uint8_t>(s);
        }
    }
}

template <typename T>
const void *norm_fn(int format) {
    switch (format) {
    case SSU_FORMAT_MXFP8: return reinterpret_cast<const void *>(&norm_kernel<T, SSU_FORMAT_MXFP8>);
    case SSU_FORMAT_MXFP4: return reinterpret_cast<const void *>(&norm_kernel<T, SSU_FORMAT_MXFP4>);
    }
    return reinterpret_cast<const void *>(&norm_kernel<T, SSU_FORMAT_SAME>);
}

}  // namespace

int launch_norm(const NormParams &p, int dtype, int format, void *stream) {
    const void *fn = dtype == SSU_F32   ? norm_fn<float>(format)
                     : dtype == SSU_F16 ? norm_fn<_Float16>(format)
                                        : norm_fn<__bf16>(format);
    NormParams pc = p;
    void *args[] = {&pc};
    return static_cast<int>(hipLaunchKernel(fn, dim3(static_cast<unsigned>(p.parts)), dim3(kNormThreads), args, 0,
                                            static_cast<hipStream_t>(stream)));
}

}  // namespace ssu
