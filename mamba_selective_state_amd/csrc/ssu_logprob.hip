// Log probabilities of given tokens with entropy, rank and the top
// alternatives (ssu_token_logprobs).
#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kLogprobThreads = 256;
constexpr int kLogprobWaves = kLogprobThreads / kWaveLanes;

// A logit's place in the order of alternatives: larger keys first. The high
// word orders the values, the low one prefers the lower index. 0 is below
// every allowed token's key.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t index) {
    if (v == 0.0f)
        v = 0.0f;  // -0 and 0 are equal
    const uint32_t b = __float_as_uint(v);
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

template <typename T>
__device__ T block_reduce(T v, T *shared, T (*f)(T, T)) {
    for (int d = 1; d < kWaveLanes; d *= 2) {
        T o;
        if constexpr (sizeof(T) == 8)
            o = static_cast<T>(__shfl_xor(static_cast<unsigned long long>(v), d));
        else
            o = __shfl_xor(v, d);
        v = f(v, o);
    }
    __syncthreads();
    if (threadIdx.x % kWaveLanes == 0)
        shared[threadIdx.x / kWaveLanes] = v;
    __syncthreads();
    v = shared[0];
    for (int w = 1; w < kLogprobWaves; w++)
        v = f(v, shared[w]);
    return v;
}
__device__ float add_f(float a, float b) { return a + b; }
__device__ int add_i(int a, int b) { return a + b; }
__device__ uint64_t max_k(uint64_t a, uint64_t b) { return a > b ? a : b; }

// One workgroup per row; the row is read once for the largest logit, once
// for the sums and once per alternative.
template <typename T>
__global__ __launch_bounds__(kLogprobThreads) void logprob_kernel(const LogprobParams p) {
    __shared__ float fsum[kLogprobWaves];
    __shared__ int isum[kLogprobWaves];
    __shared__ uint64_t ksum[kLogprobWaves];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.logits) + row * p.logits_s;
    const int32_t *mask = p.mask ? p.mask + row * p.mask_s : nullptr;
    const float temp = p.temperature ? p.temperature[row * p.temp_s] : 1.0f;
    const int64_t token =
        p.tokens_i64 ? static_cast<const int64_t *>(p.tokens)[row * p.tokens_s]
                     : static_cast<const int32_t *>(p.tokens)[row * p.tokens_s];
    auto listed = [&](int i) { return !mask || ((static_cast<uint32_t>(mask[i / 32]) >> (i % 32)) & 1u); };

    uint64_t best = 0;
    int bad = temp > 0.0f ? 0 : 1;
    for (int i = threadIdx.x; i < p.vocab; i += kLogprobThreads) {
        if (!listed(i))
            continue;
        const float v = widen(x[i]);
        if (!(v < __builtin_inff()))
            bad = 1;
        else if (v > -__builtin_inff())
            best = max_k(best, order_key(v, i));
    }
    best = block_reduce(best, ksum, max_k);
    bad = block_reduce(bad, isum, add_i);
    const float m = key_value(best);

    const bool inside = token >= 0 && token < p.vocab;
    const float mine = inside && listed(static_cast<int>(token)) ? widen(x[token]) : -__builtin_inff();
    const uint64_t mine_key = mine > -__builtin_inff() ? order_key(mine, static_cast<uint32_t>(token)) : 0;
    float s = 0.0f, t = 0.0f;
    int before = 0;
    for (int i = threadIdx.x; i < p.vocab; i += kLogprobThreads) {
        if (!listed(i))
            continue;
        const float v = widen(x[i]);
        if (!(v > -__builtin_inff()))
            continue;
        const float d = (v - m) / temp;
        const float e = expf(d);
        s += e;
        t += e > 0.0f ? e * d : 0.0f;  // d may be -inf
        before += order_key(v, i) > mine_key;
    }
    s = block_reduce(s, fsum, add_f);
    t = block_reduce(t, fsum, add_f);
    before = block_reduce(before, isum, add_i);
    const float ls = logf(s);
    if (threadIdx.x == 0) {
        const float nan = __builtin_nanf("");
        p.logprob[row] = bad ? nan : mine_key ? (mine - m) / temp - ls : -__builtin_inff();
        p.entropy[row] = bad ? nan : best ? ls - t / s : 0.0f;
        p.rank[row] = bad || !mine_key ? -1 : before;
    }
    for (int j = 0; j < p.top; j++) {
        if (threadIdx.x == 0) {
            p.top_tokens[row * p.top + j] = bad || !best ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
            p.top_logprobs[row * p.top + j] = bad    ? __builtin_nanf("")
                                              : best ? (key_value(best) - m) / temp - ls
                                                     : -__builtin_inff();
        }
        uint64_t next = 0;
        for (int i = threadIdx.x; i < p.vocab; i += kLogprobThreads) {
            if (!listed(i))
                continue;
            const float v = widen(x[i]);
            if (!(v > -__builtin_inff()))
                continue;
            const uint64_t key = order_key(v, i);
            if (key < best)
                next = max_k(next, key);
        }
        best = block_reduce(next, ksum, max_k);
    }
}

}  // namespace

int launch_logprobs(const LogprobParams &p, int dtype, void *stream) {
    const void *fn = dtype == SSU_F32   ? reinterpret_cast<const void *>(&logprob_kernel<float>)
                     : dtype == SSU_F16 ? reinterpret_cast<const void *>(&logprob_kernel<_Float16>)
                                        : reinterpret_cast<const void *>(&logprob_kernel<__bf16>);
    LogprobParams pc = p;
    void *args[] = {&pc};
    return static_cast<int>(hipLaunchKernel(fn, dim3(static_cast<unsigned>(p.rows)), dim3(kLogprobThreads), args, 0,
                                            static_cast<hipStream_t>(stream)));
}

}  // namespace ssu
