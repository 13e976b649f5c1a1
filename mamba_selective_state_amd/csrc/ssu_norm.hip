// Gated, residual-adding RMS norm (ssu_add_rms_norm): per part of a row,
//   u = x * silu(gate) + residual,  y = u * rsqrt(mean u^2 + eps) * weight.
// The bytes bound it: every input is read once, u stays in registers between the sum
// and the outputs, and the MX codes are made where y is. 16384 x 8192 bf16 with a gate, 8 groups, to MXFP8: 134 us
// (675 MB, 5.0 TB/s, a plain copy's rate); with a residual instead, to bf16, 190 us (5.6 TB/s). 256 x 4096
// with a residual to MXFP8: 4.8 us, most of it the way there and back of one access and a barrier.
// u and the sum are f32; the residual is rounded to its type when it is stored, y is made of the
// unrounded u.
#include <algorithm>

#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kNormThreads = 256;

constexpr float kLog2eHi = 1.44269504088896341f, kLog2eLo = 1.925963033500011e-8f, kLn2 = 0.693147180559945309f;

// z * sigmoid(z) to within 2 ulps for z >= -87: the codes of an MX output go by y's last bits, and the plain
// exp2(z log2 e) loses |z| / 2 of them. log2 e is taken in two parts, the reciprocal is
// refined once. A NaN stays.
__device__ __forceinline__ float silu_exact(float z) {
    const float c = __builtin_amdgcn_fmed3f(z, -87.0f, 87.0f);
    const float hi = -c * kLog2eHi;
    const float lo = fmaf(-c, kLog2eHi, -hi) - c * kLog2eLo;
    const float e = __builtin_amdgcn_exp2f(hi);
    const float d = 1.0f + fmaf(e * lo, kLn2, e);
    const float r = __builtin_amdgcn_rcpf(d);
    return z * fmaf(fmaf(-d, r, 1.0f), r, r);
}
// The same below -87, where 1 + e^-z overflows: z e^z, with 2^96 in the exponential and out of z, so that
// only the product leaves the range of normal numbers. -inf times 0 is a NaN, as in the formula.
__device__ __forceinline__ float silu_far(float z) {
#pragma clang fp contract(off)  // lo is what the rounded hi leaves: 96 must be added to that hi
    const float c = fmaxf(z, -300.0f);
    const float hi = c * kLog2eHi;
    const float lo = fmaf(c, kLog2eHi, -hi) + c * kLog2eLo;
    const float e = __builtin_amdgcn_exp2f(hi + 96.0f);
    return z * 0x1p-96f * fmaf(e * lo, kLn2, e);
}
// v times silu(z), eight at a time: one look for all of them at whether a gate lies that far out.
__device__ __forceinline__ void apply_gate(float v[8], const float z[8]) {
    float least = z[0];
#pragma unroll
    for (int j = 1; j < 8; j++)
        least = fminf(least, z[j]);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        float s = silu_exact(z[j]);
        if (least < -87.0f)
            s = z[j] < -87.0f ? silu_far(z[j]) : s;
        v[j] *= s;
    }
}

// Eight elements of a row as loaded: all of them, or the first n and zeros after.
template <typename T>
struct Raw8 {
    typedef T Vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    Vec v;
    __device__ __forceinline__ void load(const T *src) { v = *reinterpret_cast<const Vec *>(src); }
    __device__ __forceinline__ void load(const T *src, int n) {
        if (n >= 8)
            return load(src);
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = i < n ? src[i] : static_cast<T>(0.0f);
    }
};
// The same of a tensor that has the activations' type or is f32.
template <typename T>
struct Raw8Or32 {
    Raw8<T> t;
    Raw8<float> f;
    template <typename... N>
    __device__ __forceinline__ void load(const void *base, bool f32, int64_t at, N... n) {
        if (f32)
            f.load(static_cast<const float *>(base) + at, n...);
        else
            t.load(static_cast<const T *>(base) + at, n...);
    }
    __device__ __forceinline__ float get(bool f32, int i) const { return f32 ? f.v[i] : widen(t.v[i]); }
};

template <typename T, int FORMAT>
__device__ __forceinline__ void store_result(const NormParams &p, int64_t row, int at, int n, int lane, const float y[8]) {
    if constexpr (FORMAT == SSU_FORMAT_SAME) {
        store8(static_cast<T *>(p.out) + row * p.out_s + at, n, y);
    } else {
        uint32_t code[2];
        const uint32_t s = mx_block<FORMAT>(y, code);
        store_codes<FORMAT>(static_cast<uint8_t *>(p.out) + row * p.out_s, at, code);
        if (lane % 4 == 0)
            p.scales[(row * p.groups * p.part + at) / 32] = static_cast<uint8_t>(s);
    }
}
template <typename T>
__device__ __forceinline__ void store_residual(const NormParams &p, int64_t row, int at, int n, const float u[8]) {
    if (p.res_f32)
        store8(static_cast<float *>(p.residual_out) + row * p.res_out_s + at, n, u);
    else
        store8(static_cast<T *>(p.residual_out) + row * p.res_out_s + at, n, u);
}

// LANES lanes per part (16, or whole waves), each with up to NV runs of eight elements in registers.
// WHOLE: a part is a multiple of eight. Otherwise (eight or more) its last run is the part's
// last eight elements: those that the run before has are left out of the sum, and both
// lanes store the same values there. Every access is a whole one: 8192 rows of 8191 f16 with
// a residual take 124 us, and 133 with the last run's elements one by one.
template <typename T, int FORMAT, int LANES, int NV, bool WHOLE>
__global__ __launch_bounds__(LANES < kNormThreads ? kNormThreads : LANES) void norm_kernel(const NormParams p) {
    constexpr int kThreads = LANES < kNormThreads ? kNormThreads : LANES;
    constexpr int kWaves = LANES / kWaveLanes;  // per part
    const int64_t part = LANES < kNormThreads ? static_cast<int64_t>(blockIdx.x) * (kThreads / LANES) + threadIdx.x / LANES
                                              : static_cast<int64_t>(blockIdx.x);
    if (part >= p.parts)
        return;  // whole waves, or with 16 lanes whole DPP rows
    const int lane = threadIdx.x % LANES;
    const int64_t row = part / p.groups;
    const int first = static_cast<int>(part - row * p.groups) * p.part;
    const auto has = [&](int v) { return (v * LANES + lane) * 8 < p.part; };
    const auto start = [&](int v) {
        const int i = (v * LANES + lane) * 8;
        return WHOLE ? i : min(i, p.part - 8);
    };
    Raw8<T> x[NV], z[NV];
    Raw8Or32<T> r[NV], g[NV];
#pragma unroll
    for (int v = 0; v < NV; v++) {
        x[v].v = {};
        if (has(v))
            x[v].load(static_cast<const T *>(p.x) + row * p.x_s + first + start(v));
    }
    if (p.gate)
#pragma unroll
        for (int v = 0; v < NV; v++) {
            z[v].v = {};
            if (has(v))
                z[v].load(static_cast<const T *>(p.gate) + row * p.gate_s + first + start(v));
        }
    if (p.residual)
#pragma unroll
        for (int v = 0; v < NV; v++) {
            r[v].t.v = {};
            r[v].f.v = {};
            if (has(v))
                r[v].load(p.residual, p.res_f32, row * p.res_s + first + start(v));
        }
    // one run: the weights come with the rest; more: they are fetched (mostly from the caches)
    // when the inputs' registers are free
    if constexpr (NV == 1)
        if (has(0))
            g[0].load(p.weight, p.weight_f32, first + start(0));
    float u[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; v++) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            u[v][j] = widen(x[v].v[j]);
        if (p.gate) {
            float gate[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                gate[j] = widen(z[v].v[j]);
            apply_gate(u[v], gate);
        }
        if (p.residual)
#pragma unroll
            for (int j = 0; j < 8; j++)
                u[v][j] += r[v].get(p.res_f32, j);
        const int before = WHOLE ? 0 : (v * LANES + lane) * 8 - start(v);  // more than 8 where there is no run
#pragma unroll
        for (int j = 0; j < 8; j++)
            ss = j < before ? ss : fmaf(u[v][j], u[v][j], ss);
    }
    ss = LANES == 16 ? row16_sum(ss) : wave64_sum(ss);
    if constexpr (kWaves > 1) {
        __shared__ float sums[kWaves];
        if (threadIdx.x % kWaveLanes == 0)
            sums[threadIdx.x / kWaveLanes] = ss;
        __syncthreads();
        ss = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++)
            ss += sums[w];
    }
    const float scale = 1.0f / sqrtf(ss / static_cast<float>(p.part) + p.eps);
#pragma unroll
    for (int v = 0; v < NV; v++) {
        if (!has(v))
            break;
        const int at = first + start(v);
        if (p.residual)
            store_residual<T>(p, row, at, 8, u[v]);
        if constexpr (NV > 1)
            g[v].load(p.weight, p.weight_f32, at);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; j++)
            y[j] = u[v][j] * scale * g[v].get(p.weight_f32, j);
        store_result<T, FORMAT>(p, row, at, 8, lane, y);
    }
}

// Parts that no workgroup's registers hold: the inputs are read again for the outputs (2048
// rows of 65536 bf16 with a residual: 284 us, 3.8 TB/s counting each byte once). Parts of
// fewer than eight elements: one wave each.
constexpr int kLongThreads = 1024;
template <typename T, int FORMAT>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(const NormParams p) {
    __shared__ float sums[kLongThreads / kWaveLanes];
    const int64_t part = blockIdx.x;
    const int64_t row = part / p.groups;
    const int first = static_cast<int>(part - row * p.groups) * p.part;
    const int tid = threadIdx.x, threads = blockDim.x;
    auto load_u = [&](int i, int n, float u[8]) {
        Raw8<T> x;
        x.load(static_cast<const T *>(p.x) + row * p.x_s + first + i, n);
#pragma unroll
        for (int j = 0; j < 8; j++)
            u[j] = widen(x.v[j]);
        if (p.gate) {
            x.load(static_cast<const T *>(p.gate) + row * p.gate_s + first + i, n);
            float gate[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                gate[j] = widen(x.v[j]);
            apply_gate(u, gate);
        }
        if (p.residual) {
            Raw8Or32<T> r;
            r.load(p.residual, p.res_f32, row * p.res_s + first + i, n);
#pragma unroll
            for (int j = 0; j < 8; j++)
                u[j] += r.get(p.res_f32, j);
        }
    };
    float ss = 0.0f;
    for (int i = tid * 8; i < p.part; i += threads * 8) {
        float u[8];
        load_u(i, p.part - i, u);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++)
            s = fmaf(u[j], u[j], s);
        ss += s;
    }
    ss = wave64_sum(ss);
    if (tid % kWaveLanes == 0)
        sums[tid / kWaveLanes] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int w = 0; w < threads / kWaveLanes; w++)
        ss += sums[w];
    const float scale = 1.0f / sqrtf(ss / static_cast<float>(p.part) + p.eps);
    for (int i = tid * 8; i < p.part; i += threads * 8) {
        const int n = p.part - i;
        float u[8];
        load_u(i, n, u);
        Raw8Or32<T> g;
        g.load(p.weight, p.weight_f32, first + i, n);
        if (p.residual)
            store_residual<T>(p, row, first + i, n, u);
#pragma unroll
        for (int j = 0; j < 8; j++)
            u[j] = u[j] * scale * g.get(p.weight_f32, j);
        store_result<T, FORMAT>(p, row, first + i, n, tid, u);
    }
}

struct NormShape {
    int lanes, nv;  // nv 0: the long kernel
};

// Lanes per part. Many elements: the fewest lanes that keep a part in registers (no barrier
// for up to 2048). Few: the time of one part is the time of the call, so one run per lane up to
// 2048 elements, two for up to 4096, then as many lanes as a workgroup has. Kernel times in us, bf16
// with a residual:
//   256 x 2048: 64 lanes 4.27, 256 lanes 2.65; 1024 x 2048: 5.17, 4.04; 4096 x 2048: 10.8, 12.3
//   256 x 8192: 256 lanes 5.16, 1024 lanes 4.33; 1024 x 8192: 10.8, 13.3
//   256 x 4096: 256 lanes 4.70, 1024 lanes 4.24; 900 x 4096: 9.3, 10.9; 900 x 2561: 6.7, 8.3 (so for
//     up to 4096 the two cross between 256 and 900 rows, where the rule takes 256 lanes throughout)
//   65536 x 128: 16 lanes 13.0, 64 lanes 23.7; 65536 x 512: 64 lanes 40, 256 lanes 57
NormShape shape_for(int64_t parts, int part) {
    if (part < 8)
        return {kWaveLanes, 0};
    const int runs = (part + 7) / 8;
    constexpr NormShape kShapes[] = {{16, 1},  {64, 1},  {64, 2},   {64, 4},   {256, 1},
                                     {256, 2}, {256, 4}, {1024, 1}, {1024, 2}, {1024, 4}};
    const bool many = parts * part >= (1 << 22);
    for (const NormShape &s : kShapes)
        if (runs <= s.lanes * s.nv && (many || s.nv == 1 || s.lanes * s.nv == 512 || s.lanes == 1024))
            return s;
    return {kLongThreads, 0};
}

template <typename T, int FORMAT, bool WHOLE>
const void *norm_fn(NormShape s) {
    switch (s.lanes * 8 + s.nv) {
    case 16 * 8 + 1: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 16, 1, WHOLE>);
    case 64 * 8 + 1: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 64, 1, WHOLE>);
    case 64 * 8 + 2: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 64, 2, WHOLE>);
    case 64 * 8 + 4: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 64, 4, WHOLE>);
    case 256 * 8 + 1: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 256, 1, WHOLE>);
    case 256 * 8 + 2: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 256, 2, WHOLE>);
    case 256 * 8 + 4: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 256, 4, WHOLE>);
    case 1024 * 8 + 1: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 1024, 1, WHOLE>);
    case 1024 * 8 + 2: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 1024, 2, WHOLE>);
    case 1024 * 8 + 4: return reinterpret_cast<const void *>(&norm_kernel<T, FORMAT, 1024, 4, WHOLE>);
    }
    return reinterpret_cast<const void *>(&norm_long_kernel<T, FORMAT>);
}
template <typename T>
const void *norm_fn(int format, bool whole, NormShape s) {
    return format == SSU_FORMAT_MXFP8   ? norm_fn<T, SSU_FORMAT_MXFP8, true>(s)
           : format == SSU_FORMAT_MXFP4 ? norm_fn<T, SSU_FORMAT_MXFP4, true>(s)
           : whole                      ? norm_fn<T, SSU_FORMAT_SAME, true>(s)
                                        : norm_fn<T, SSU_FORMAT_SAME, false>(s);
}

}  // namespace

int launch_norm(const NormParams &p, int dtype, int format, void *stream) {
    const NormShape s = shape_for(p.parts, p.part);
    const bool whole = p.part % 8 == 0;
    const void *fn = dtype == SSU_F32   ? norm_fn<float>(format, whole, s)
                     : dtype == SSU_F16 ? norm_fn<_Float16>(format, whole, s)
                                        : norm_fn<__bf16>(format, whole, s);
    const int per = s.nv && s.lanes < kNormThreads ? kNormThreads / s.lanes : 1;
    NormParams pc = p;
    void *args[] = {&pc};
    return launch_groups(fn, (p.parts + per - 1) / per, s.lanes * per, args, stream);
}

}  // namespace ssu
