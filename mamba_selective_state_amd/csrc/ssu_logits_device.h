// Device helpers of the kernels that scan rows of logits (ssu_logprob.hip, ssu_beam.hip): the order
// of a row's tokens, and the first of them that a wave has seen.
#pragma once

#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kVec = 8;                      // logits per lane and access
constexpr float kLowest = -3.402823466e38f;  // the lowest finite value

// A logit's place in the order of alternatives: larger keys first. The high
// word orders the values, the low one prefers the lower index. 0 is below
// every allowed token's key.
__device__ __forceinline__ uint32_t order_word(float v) {
    const uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);  // -0 and 0 are equal
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(uint32_t word, uint32_t index) {
    return (static_cast<uint64_t>(word) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float word_value(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }
__device__ __forceinline__ float key_value(uint64_t key) { return word_value(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ int32_t key_index(uint64_t key) {
    return static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}
// The next float below and above a finite value.
__device__ __forceinline__ float next_below(float v) {
    const uint32_t b = __float_as_uint(v);
    return v == 0.0f ? __uint_as_float(0x80000001u) : __uint_as_float(v > 0.0f ? b - 1 : b + 1);
}
__device__ __forceinline__ float next_above(float v) { return -next_below(-v); }

// Over the wave, the same in every lane; all lanes must be active.
__device__ __forceinline__ float wave_max(float v) {
    const int m = __float_as_int(group_max<16>(v));
    return fmaxf(fmaxf(__int_as_float(__builtin_amdgcn_readlane(m, 0)), __int_as_float(__builtin_amdgcn_readlane(m, 16))),
                 fmaxf(__int_as_float(__builtin_amdgcn_readlane(m, 32)), __int_as_float(__builtin_amdgcn_readlane(m, 48))));
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < kWaveLanes; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

// The first tokens of what a wave has seen, in order, one per lane: lane i holds the i-th
// (lanes from `top` on hold what was pushed out). A logit enters only if it stands before the
// `top`-th, so after the first access hardly any does.
struct Candidates {
    uint64_t key;    // this lane's token; 0: none
    uint64_t floor;  // keys above it enter: the top-th token's, or a bound below it; uniform
    float gate;      // logits below it do not enter

    // After `key` has changed.
    __device__ __forceinline__ void raise(int top) {
        const uint64_t k = (static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(key >> 32), top - 1)) << 32) |
                           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(key), top - 1));
        if (k != 0) {
            floor = k;
            // an equal logit at a lower index of the same access may still enter
            gate = fmaxf(gate, key_value(k));
        }
    }
    __device__ __forceinline__ void insert(uint64_t k, int top, int lane) {
        const uint64_t behind = __ballot(k > key);
        if (behind == 0)
            return;
        const int at = __builtin_ctzll(behind);  // lanes are in order: all from here on move up
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(key >> 32), 0x138, 0xF, 0xF, false);  // wave_shr:1
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(key), 0x138, 0xF, 0xF, false);
        const uint64_t left = (static_cast<uint64_t>(hi) << 32) | lo;
        key = lane > at ? left : lane == at ? k : key;
        raise(top);
    }
    // The first access's logits, while nothing has entered: those at or above the gate are put in
    // order together, through `list` (kList keys of LDS). False, and nothing done, where they are
    // too many.
    static constexpr int kList = 256;
    __device__ __forceinline__ bool first(const float x[kVec], uint32_t at, int top, int lane, uint64_t *list) {
        constexpr int kMost = kList / 2;
        int n = 0;
        uint64_t pass[kVec];
#pragma unroll
        for (int i = 0; i < kVec; i++) {
            pass[i] = __ballot(x[i] >= gate && x[i] < __builtin_inff());
            n += __popcll(pass[i]);
        }
        if (n > kMost)
            return false;
        int to = 0;
#pragma unroll
        for (int i = 0; i < kVec; i++) {
            const int mine = to + __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(pass[i] >> 32),
                                                            __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(pass[i]), 0));
            if ((pass[i] >> lane) & 1)
                list[mine] = order_key(order_word(x[i]), at + i);
            to += __popcll(pass[i]);
        }
        // up to the next multiple of eight, keys that stand behind all
        if (lane < 8 && n + lane < kMost)
            list[n + lane] = 0;
        list[kMost + lane] = 0;
        wave_lds_fence();
        const uint64_t a = list[lane], b = list[64 + lane];
        int ra = 0, rb = 0;
        for (int j = 0; j < n; j += 8)
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const uint64_t o = list[j + q];
                ra += o > a;
                rb += o > b;
            }
        wave_lds_fence();
        if (lane < n && ra < kWaveLanes)
            list[kMost + ra] = a;
        if (64 + lane < n && rb < kWaveLanes)
            list[kMost + rb] = b;
        wave_lds_fence();
        key = list[kMost + lane];
        raise(top);
        return true;
    }
    // An access's logits (destroyed), the lane's first index `at`: the lanes' largest ones are
    // offered and taken out until none is left that could enter.
    __device__ __forceinline__ void offer(float x[kVec], uint32_t at, int top, int lane) {
        while (true) {
            float best = x[0], second = -__builtin_inff();
            uint32_t i = 0;
#pragma unroll
            for (int j = 1; j < kVec; j++) {
                const bool larger = x[j] > best;
                second = fmaxf(second, larger ? best : x[j]);
                best = larger ? x[j] : best;
                i = larger ? j : i;
            }
            const uint64_t k = order_key(order_word(best), at + i);
            const bool pass = best >= gate && best < __builtin_inff() && k > floor;
            uint64_t todo = __ballot(pass);
            if (todo == 0)
                return;
            while (todo) {
                const int from = __builtin_ctzll(todo);
                insert((static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(k >> 32), from)) << 32) |
                           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(k), from)),
                       top, lane);
                todo &= todo - 1;
                todo &= __ballot(k > floor);
            }
            if (__ballot(second >= gate) == 0)
                return;
#pragma unroll
            for (int j = 0; j < kVec; j++)
                x[j] = pass && i == static_cast<uint32_t>(j) ? -__builtin_inff() : x[j];
        }
    }
    // A bound before anything has entered, from each lane's largest logit: at least `top` lanes
    // are at or above it (their words' leading 16 bits, found bit by bit).
    __device__ __forceinline__ void bound(float best, int top) {
        const uint32_t w = order_word(best);
        uint32_t b = 0;
#pragma unroll
        for (int bit = 31; bit >= 16; bit--) {
            const uint32_t t = b | (1u << bit);
            if (__popcll(__ballot(w >= t)) >= top)
                b = t;
        }
        if (b > 0x007FFFFFu) {  // above -inf's word
            floor = static_cast<uint64_t>(b) << 32;  // behind every key of that value
            gate = word_value(b);
        }
    }
};

}  // namespace
}  // namespace ssu
