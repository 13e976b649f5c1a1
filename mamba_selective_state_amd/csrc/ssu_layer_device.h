// Device helpers shared by the layer operators' kernels: rows read eight
// elements at a time, and eight fp32 values to their MX codes.
#pragma once

#include <hip/hip_runtime.h>

#include "ssu_device.h"
#include "ssu_layer.h"

namespace ssu {
namespace {

// Whether one launch takes them.
inline bool groups_fit(int64_t groups, int threads) { return groups <= static_cast<int64_t>(UINT32_MAX) / threads; }

inline int launch_groups(const void *fn, int64_t groups, int threads, void **args, void *stream, unsigned lds_bytes = 0) {
    if (!groups_fit(groups, threads))
        return kTooManyWorkItems;
    return static_cast<int>(hipLaunchKernel(fn, dim3(static_cast<unsigned>(groups)), dim3(static_cast<unsigned>(threads)), args, lds_bytes,
                                            static_cast<hipStream_t>(stream)));
}

// Eight consecutive elements at any element-aligned address: gfx950's global
// loads take unaligned addresses, so one 16-byte (f32: two) access serves
// every row stride.
template <typename T>
__device__ __forceinline__ void load8(const T *src, float v[8]) {
    typedef T Vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    const Vec r = *reinterpret_cast<const Vec *>(src);
#pragma unroll
    for (int i = 0; i < 8; i++)
        v[i] = widen(r[i]);
}
template <typename T>
__device__ __forceinline__ void store8(T *dst, const float v[8]) {
    typedef T Vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    Vec r;
#pragma unroll
    for (int i = 0; i < 8; i++)
        r[i] = narrow<T>(v[i]);
    *reinterpret_cast<Vec *>(dst) = r;
}

// The first `n` (up to 8) of them.
template <typename T>
__device__ __forceinline__ void store8(T *dst, int n, const float v[8]) {
    if (n >= 8)
        return store8(dst, v);
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (i < n)
            dst[i] = narrow<T>(v[i]);
}

// Between a wave's LDS writes and its other lanes' reads of them (or the reverse): the hardware keeps
// a wave's LDS accesses in order, and the fences make the compiler do so across lanes.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Sum over the wave, the same in every lane; all lanes must be active.
__device__ __forceinline__ float wave64_sum(float v) {
    const int s = __float_as_int(row16_sum(v));
    return (__int_as_float(__builtin_amdgcn_readlane(s, 0)) + __int_as_float(__builtin_amdgcn_readlane(s, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(s, 32)) + __int_as_float(__builtin_amdgcn_readlane(s, 48)));
}

// Codes of four finite values over 2^k (see e4m3_codes4 and e2m1_codes4, whose care for NaN
// elements a finite block does without).
template <int FORMAT>
__device__ __forceinline__ uint32_t finite_codes4(const float v[4], int k) {
    const float X = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    if constexpr (FORMAT == SSU_FORMAT_MXFP8) {
        const float lim = 448.0f * X;  // the conversion makes NaN of what lies beyond
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            c[i] = __builtin_amdgcn_fmed3f(v[i], -lim, lim);
        typedef short short2_t __attribute__((ext_vector_type(2)));
        short2_t r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[0], c[1], X, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c[2], c[3], X, true);
        return __builtin_bit_cast(uint32_t, r);
    } else {
        uint32_t r = 0;  // the conversion saturates
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], X, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], X, 1);
        return r & 0xFFFFu;
    }
}

// Four consecutive lanes hold a block of 32 values, eight each; every lane
// gives the codes of its eight (MXFP8: two words, MXFP4: the first) and the
// block's scale byte. The largest magnitude is taken over the bit patterns, where
// infinities and NaNs are the largest: such a block takes the scale byte
// 0xFF and zero codes. All four lanes must be active.
template <int FORMAT>
__device__ __forceinline__ uint32_t mx_block(const float v[8], uint32_t code[2]) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; i++)
        a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    a = max(a, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(a), 0xB1, 0xF, 0xF, false)));
    a = max(a, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(a), 0x4E, 0xF, 0xF, false)));
    const float amax = __uint_as_float(a);
    const int k = FORMAT == SSU_FORMAT_MXFP8 ? mx8_exponent(amax) : mx4_exponent(amax);
    code[0] = finite_codes4<FORMAT>(v, k);
    code[1] = finite_codes4<FORMAT>(v + 4, k);
    if constexpr (FORMAT == SSU_FORMAT_MXFP4) {
        code[0] |= code[1] << 16;
        code[1] = 0;
    }
    const bool finite = a < 0x7F800000u;
    code[0] = finite ? code[0] : 0;
    code[1] = finite ? code[1] : 0;
    return finite ? static_cast<uint32_t>(k + 127) : 0xFFu;
}

// Stores a lane's eight codes; `at` is its first value's index in the row.
template <int FORMAT>
__device__ __forceinline__ void store_codes(uint8_t *row, int64_t at, const uint32_t code[2]) {
    if constexpr (FORMAT == SSU_FORMAT_MXFP8)
        *reinterpret_cast<u32x2 *>(row + at) = u32x2{code[0], code[1]};
    else
        *reinterpret_cast<uint32_t *>(row + at / 2) = code[0];
}

}  // namespace
}  // namespace ssu
