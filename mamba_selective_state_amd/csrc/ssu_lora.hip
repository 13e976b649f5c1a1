// Low-rank adapters of many requests beside a shared projection (ssu_add_lora):
//   h = x A_i^T (down: k to rank),   y += (scale_i h) B_i^T (up: rank to n),   i the row's adapter.
//
// Rows of one adapter are worked on together, so that each adapter's weights are read once for up to a tile of rows.
// Which rows these are is found on the device: lora_plan makes lists of tiles (an adapter and a run of `perm`).
// Up to kSelfRows rows, the down kernel's workgroups look their rows up for themselves, and one more workgroup makes the
// plan for the up kernel in the meantime: two launches. More rows: plan, down, up.
//
// Rows of other adapters never meet a weight, not even times zero: what one adapter's weights hold (NaN, infinity) stays with
// its rows. h is f32 in the workspace; the up kernel splits 16-bit types' h into two summands of that type, hi + lo,
// which go through the matrix instructions one after the other against the same weights: h keeps 16 (bf16) or 22
// (f16) bits, where one of that type would keep 8 or 11. The up kernel waits for y, not for products, so this is free.
//
// Operand layout of the 16-row instructions: lane l holds row l % 16 of its operand and the k values of group
// l / 16; the result's lane l holds rows 4 (l / 16) .. + 3 of the first operand for row l % 16 of the second. The
// weights go first, so that a lane has four neighbouring outputs of one row.
#include <algorithm>

#include "ssu_layer_device.h"

namespace ssu {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct Mx8 {};  // rows as MXFP8 or MXFP4 codes and scales
struct Mx4 {};

// Eight k values of one row.
template <typename T>
struct Frag {
    typedef T V __attribute__((ext_vector_type(8)));
    V v;
};

// 32 values of k: lane group g's eight are 8 g .. 8 g + 7 of both operands.
__device__ __forceinline__ f32x4 mma(const Frag<__bf16> &a, const Frag<__bf16> &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<_Float16> &a, const Frag<_Float16> &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float> &a, const Frag<float> &b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 8; i++)  // one value of each group at a time
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
}

template <typename T>
__device__ __forceinline__ Frag<T> zero_frag() {
    Frag<T> f;
#pragma unroll
    for (int i = 0; i < 8; i++)
        f.v[i] = static_cast<T>(0.0f);
    return f;
}
template <typename T>
__device__ __forceinline__ Frag<T> load_frag(const T *p) {
    typedef T V __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    Frag<T> f;
    f.v = *reinterpret_cast<const V *>(p);
    return f;
}
// The first `n` of them (any n), 0 for the rest.
template <typename T>
__device__ __forceinline__ Frag<T> load_frag(const T *p, int n) {
    if (n >= 8)
        return load_frag(p);
    Frag<T> f = zero_frag<T>();
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (i < n)
            f.v[i] = p[i];
    return f;
}

// ---------------------------------------------------------------- the plan

constexpr int kDownRows = 32;  // rows of a down tile
constexpr int kUpRows = 128;   // rows of an up tile
constexpr int kSelfRows = 2048;

struct Tile {
    int32_t adapter, first, count, unused;  // rows perm[first .. first + count)
};
struct LoraPlan {
    int32_t *counts;  // up tiles, down tiles
    Tile *up, *down;
    int32_t *perm;
    float *h;  // [slices][rows][rank, padded]
};

__device__ __forceinline__ int adapter_of(const LoraParams &p, int row) {
    const int64_t v = p.ids_i64 ? static_cast<const int64_t *>(p.ids)[row * p.ids_s] : static_cast<const int32_t *>(p.ids)[row * p.ids_s];
    return v >= 0 && v < p.adapters ? static_cast<int>(v) : -1;
}

// Adds one to counter[id] for every lane with an id (>= 0); the lane's number among them. One addition
// where the wave's ids agree, as in a request's run of tokens: the counter would serve its lanes one at a time.
__device__ __forceinline__ int draw_number(int *counter, int id, int lane) {
    const uint64_t live = __ballot(id >= 0);
    if (live == 0)
        return 0;
    const int first = __builtin_ctzll(live);
    const int lead = __builtin_amdgcn_readlane(id, first);
    const uint64_t same = __ballot(id == lead);
    if (same == live) {
        int base = 0;
        if (lane == first)
            base = atomicAdd(&counter[lead], static_cast<int>(__popcll(live)));
        base = __builtin_amdgcn_readlane(base, first);
        return base + __popcll(live & ((1ull << lane) - 1));
    }
    return id >= 0 ? atomicAdd(&counter[id], 1) : 0;
}

// By one workgroup of THREADS; `hist`: `adapters` counters in LDS. The order of an adapter's rows may differ from call to call;
// a row's result does not depend on it.
template <int THREADS>
__device__ void make_plan(const LoraParams &p, const LoraPlan &plan, int *hist) {
    constexpr int kWaves = THREADS / kWaveLanes;
    __shared__ int sums[3][kWaves];
    const int t = threadIdx.x, lane = t % kWaveLanes, wave = t / kWaveLanes;
    for (int i = t; i < p.adapters; i += THREADS)
        hist[i] = 0;
    __syncthreads();
    const int rounds = (p.rows + THREADS - 1) / THREADS;
    for (int i = 0; i < rounds; i++) {
        const int row = i * THREADS + t;
        draw_number(hist, row < p.rows ? adapter_of(p, row) : -1, lane);
    }
    __syncthreads();
    // a run of adapters for each thread: rows, up tiles and down tiles before it
    const int per = (p.adapters + THREADS - 1) / THREADS;
    const int begin = min(t * per, p.adapters), end = min(begin + per, p.adapters);
    int own[3] = {0, 0, 0};
    for (int a = begin; a < end; a++) {
        own[0] += hist[a];
        own[1] += (hist[a] + kUpRows - 1) / kUpRows;
        own[2] += (hist[a] + kDownRows - 1) / kDownRows;
    }
    int at[3];
#pragma unroll
    for (int q = 0; q < 3; q++) {
        int v = own[q];
#pragma unroll
        for (int d = 1; d < kWaveLanes; d *= 2) {
            const int o = __shfl_up(v, d);
            v += lane >= d ? o : 0;
        }
        if (lane == kWaveLanes - 1)
            sums[q][wave] = v;
        at[q] = v - own[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 3; q++)
        for (int w = 0; w < kWaves; w++)
            at[q] += w < wave ? sums[q][w] : 0;
    if (t == THREADS - 1) {
        plan.counts[0] = at[1] + own[1];
        plan.counts[1] = at[2] + own[2];
    }
    for (int a = begin; a < end; a++) {
        const int n = hist[a];
        for (int i = 0; i < n; i += kUpRows)
            plan.up[at[1]++] = {a, at[0] + i, min(kUpRows, n - i), 0};
        for (int i = 0; i < n; i += kDownRows)
            plan.down[at[2]++] = {a, at[0] + i, min(kDownRows, n - i), 0};
        hist[a] = at[0];
        at[0] += n;
    }
    __syncthreads();
    for (int i = 0; i < rounds; i++) {
        const int row = i * THREADS + t;
        const int id = row < p.rows ? adapter_of(p, row) : -1;
        const int to = draw_number(hist, id, lane);
        if (id >= 0)
            plan.perm[to] = row;
    }
}

constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void lora_plan_kernel(const LoraParams p, const LoraPlan plan) {
    extern __shared__ int dynamic[];
    make_plan<kPlanThreads>(p, plan, dynamic);
}

// ---------------------------------------------------------------- down

constexpr int kDownThreads = 512;
constexpr int kDownWaves = kDownThreads / kWaveLanes;

// Rows of x as operands of type T.
template <typename T, typename SRC>
struct XRow {
    const SRC *row;
    __device__ __forceinline__ XRow(const LoraParams &p, int64_t r) : row(static_cast<const SRC *>(p.x) + r * p.x_s) {}
    __device__ __forceinline__ Frag<T> load(int at, int n) const { return load_frag<T>(row + at, n); }
    __device__ __forceinline__ Frag<T> load(int at) const { return load_frag<T>(row + at); }
};
// Codes: exact in bf16, which has their four bits and, but for its ends, their scales' range.
template <>
struct XRow<__bf16, Mx8> {
    const uint8_t *codes, *scales;
    __device__ __forceinline__ XRow(const LoraParams &p, int64_t r)
        : codes(static_cast<const uint8_t *>(p.x) + r * p.x_s), scales(p.x_scale + r * p.xs_s) {}
    __device__ __forceinline__ Frag<__bf16> load(int at) const {
        typedef u32x2 Any2 __attribute__((aligned(1)));
        const u32x2 c = *reinterpret_cast<const Any2 *>(codes + at);
        const uint32_t s = scales[at / 32];
        const float scale = mx8_scale(s);
        Frag<__bf16> f;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2 lo = e4m3_pair<false>(c[i], scale), hi = e4m3_pair<true>(c[i], scale);
            const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
            for (int j = 0; j < 4; j++)
                f.v[4 * i + j] = narrow<__bf16>(s == 255 ? __builtin_nanf("") : v[j]);
        }
        return f;
    }
    __device__ __forceinline__ Frag<__bf16> load(int at, int n) const { return n > 0 ? load(at) : zero_frag<__bf16>(); }
};
template <>
struct XRow<__bf16, Mx4> {
    const uint8_t *codes, *scales;
    __device__ __forceinline__ XRow(const LoraParams &p, int64_t r)
        : codes(static_cast<const uint8_t *>(p.x) + r * p.x_s), scales(p.x_scale + r * p.xs_s) {}
    __device__ __forceinline__ Frag<__bf16> load(int at) const {
        typedef uint32_t Any1 __attribute__((aligned(1)));
        const uint32_t c = *reinterpret_cast<const Any1 *>(codes + at / 2);
        const uint32_t s = scales[at / 32];
        const float scale = mx8_scale(s);
        const float2 v[4] = {e2m1_pair<0>(c, scale), e2m1_pair<1>(c, scale), e2m1_pair<2>(c, scale), e2m1_pair<3>(c, scale)};
        Frag<__bf16> f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f.v[2 * j] = narrow<__bf16>(s == 255 ? __builtin_nanf("") : v[j].x);
            f.v[2 * j + 1] = narrow<__bf16>(s == 255 ? __builtin_nanf("") : v[j].y);
        }
        return f;
    }
    __device__ __forceinline__ Frag<__bf16> load(int at, int n) const { return n > 0 ? load(at) : zero_frag<__bf16>(); }
};

// h of up to 16 XF rows of one adapter over values [begin, end) of k. `row_of`(i): the i-th row. The waves take
// turns at steps of 32 and join their sums in LDS, in a fixed order.
template <typename T, typename SRC, int RF, int XF, typename F>
__device__ __forceinline__ void down_tile(const LoraParams &p, int adapter, int count, int begin, int end, float *h, f32x4 *sums, F &&row_of) {
    constexpr int kGroup = 4;  // fragments joined at a time
    const int lane = threadIdx.x % kWaveLanes, wave = threadIdx.x / kWaveLanes;
    const int r = lane % 16, g = lane / 16;
    const T *a[RF];
#pragma unroll
    for (int f = 0; f < RF; f++)  // rank rows past the end read the last one; what they give is not used
        a[f] = static_cast<const T *>(p.a) + adapter * p.a_l + min(f * 16 + r, p.rank - 1) * p.a_r;
    const XRow<T, SRC> x0(p, row_of(min(r, count - 1)));
    const XRow<T, SRC> x1(p, XF > 1 ? row_of(min(16 + r, count - 1)) : 0);
    f32x4 acc[XF][RF] = {};
    auto step = [&](auto load_x, auto load_a) {
        Frag<T> x[XF], w[RF];
        x[0] = load_x(x0);
        if constexpr (XF > 1)
            x[1] = load_x(x1);
#pragma unroll
        for (int f = 0; f < RF; f++)
            w[f] = load_a(a[f]);
#pragma unroll
        for (int i = 0; i < XF; i++)
#pragma unroll
            for (int f = 0; f < RF; f++)
                acc[i][f] = mma(w[f], x[i], acc[i][f]);
    };
    int at = begin + wave * 32;
#pragma unroll 2
    for (; at + 32 <= end; at += kDownWaves * 32)
        step([&](const XRow<T, SRC> &x) { return x.load(at + 8 * g); }, [&](const T *w) { return load_frag(w + at + 8 * g); });
    if (at < end) {
        const int n = end - at - 8 * g;
        step([&](const XRow<T, SRC> &x) { return x.load(at + 8 * g, n); }, [&](const T *w) { return load_frag(w + at + 8 * g, n); });
    }
    constexpr int kFrags = XF * RF;
#pragma unroll
    for (int f0 = 0; f0 < kFrags; f0 += kGroup) {
        constexpr int kIn = kFrags < kGroup ? kFrags : kGroup;
        __syncthreads();
#pragma unroll
        for (int f = 0; f < kIn; f++)
            sums[(wave * kIn + f) * 64 + lane] = acc[(f0 + f) / RF][(f0 + f) % RF];
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < kIn * 64) {
            const int f = f0 + wave;
            f32x4 v = sums[wave * 64 + lane];
#pragma unroll
            for (int w = 1; w < kDownWaves; w++)
                v += sums[(w * kIn + wave) * 64 + lane];
            const int row = f / RF * 16 + r;
            if (row < count)
                *reinterpret_cast<f32x4 *>(h + static_cast<int64_t>(row_of(row)) * (RF * 16) + f % RF * 16 + 4 * g) = v;
        }
    }
}

// SELF: a workgroup for each (adapter or leading row, slice of k) looks its rows up, the first workgroup makes the plan.
template <typename T, typename SRC, int RF, bool SELF>
__global__ __launch_bounds__(kDownThreads) void lora_down_kernel(const LoraParams p, const LoraPlan plan) {
    extern __shared__ int dynamic[];
    __shared__ f32x4 sums[kDownWaves * 4 * 64];
    __shared__ int mine[SELF ? kSelfRows : 1];
    __shared__ int found;
    int id = static_cast<int>(blockIdx.x);
    if constexpr (SELF) {
        if (id == 0) {
            make_plan<kDownThreads>(p, plan, dynamic);
            return;
        }
        id--;
    }
    const int slice = id % p.slices;
    const int begin = slice * p.slice, end = min(p.k, begin + p.slice);
    float *h = plan.h + static_cast<int64_t>(slice) * p.rows * (RF * 16);
    if constexpr (SELF) {
        const int lane = threadIdx.x % kWaveLanes;
        int adapter = id / p.slices, from = 0;
        if (p.rows < p.adapters) {  // the row's adapter, if no row before it has it
            from = adapter;
            adapter = adapter_of(p, from);
            if (adapter < 0)
                return;
        }
        if (threadIdx.x == 0)
            found = 0;
        __syncthreads();
        bool earlier = false;
        for (int i = 0; i < p.rows; i += kDownThreads) {
            const int row = i + threadIdx.x;
            const bool is = row < p.rows && adapter_of(p, row) == adapter;
            earlier = earlier || (is && row < from);
            const uint64_t which = __ballot(is);
            int base = 0;
            if (lane == 0 && which != 0)
                base = atomicAdd(&found, static_cast<int>(__popcll(which)));
            base = __builtin_amdgcn_readfirstlane(base);
            if (is)
                mine[base + __popcll(which & ((1ull << lane) - 1))] = row;
        }
        if (__syncthreads_or(earlier))
            return;
        const int n = found;
        for (int i = 0; i < n; i += 16)
            down_tile<T, SRC, RF, 1>(p, adapter, min(16, n - i), begin, end, h, sums, [&](int j) { return mine[i + j]; });
    } else {
        const int tile = id / p.slices;
        if (tile >= plan.counts[1])
            return;
        const Tile t = plan.down[tile];
        down_tile<T, SRC, RF, kDownRows / 16>(p, t.adapter, t.count, begin, end, h, sums, [&](int j) { return plan.perm[t.first + j]; });
    }
}

// ---------------------------------------------------------------- up

constexpr int kUpThreads = 256;
constexpr int kUpWaves = kUpThreads / kWaveLanes;
constexpr int kUpCols = 64;  // of a wave

// Eight f32 as one operand, or as two whose sum they are to twice its digits.
template <typename T>
__device__ __forceinline__ void split_value(float v, T *hi, T *lo) {
    *hi = narrow<T>(v);
    const float w = widen(*hi);
    *lo = narrow<T>(fabsf(w) < __builtin_inff() ? v - w : 0.0f);
}

template <typename T, int R>
__global__ __launch_bounds__(kUpThreads) void lora_up_kernel(const LoraParams p, const LoraPlan plan) {
    constexpr int KB = R < 32 ? 1 : R / 32;  // operands of 32 along the rank
    constexpr bool kSplit = sizeof(T) == 2;
    constexpr bool kBoth = kSplit && R == 16;  // hi and lo fill one operand
    const int lane = threadIdx.x % kWaveLanes, wave = threadIdx.x / kWaveLanes;
    const int r = lane % 16, g = lane / 16;
    const int blocks = (p.n + kUpWaves * kUpCols - 1) / (kUpWaves * kUpCols);
    const int64_t items = static_cast<int64_t>(plan.counts[0]) * blocks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const Tile t = plan.up[item / blocks];
        const int n0 = static_cast<int>(item % blocks) * (kUpWaves * kUpCols) + wave * kUpCols;
        if (n0 >= p.n)
            continue;
        // fragment f's row i is output n0 + 32 (f / 2) + 8 (i / 4) + 4 (f % 2) + i % 4: a lane's results of
        // two fragments are eight neighbours
        Frag<T> w[4][KB];
#pragma unroll
        for (int f = 0; f < 4; f++) {
            const int at = min(n0 + 32 * (f / 2) + 8 * (r / 4) + 4 * (f % 2) + r % 4, p.n - 1);
            const T *row = static_cast<const T *>(p.b) + t.adapter * p.b_l + at * p.b_n;
#pragma unroll
            for (int kb = 0; kb < KB; kb++) {
                const int k0 = kBoth ? 8 * (g % 2) : 32 * kb + 8 * g;
                w[f][kb] = load_frag(row + k0, p.rank - k0);
            }
        }
        const float scale = p.scale ? p.scale[t.adapter * p.scale_s] : 1.0f;
        for (int c = 0; c < t.count; c += 16) {
            const int row = plan.perm[t.first + min(c + r, t.count - 1)];
            T *y = static_cast<T *>(p.y) + row * p.y_s + n0 + 8 * g;
            float v[2][8] = {};
#pragma unroll
            for (int s = 0; s < 2; s++) {
                const int left = p.n - n0 - 32 * s - 8 * g;
                if (left >= 8) {
                    load8(y + 32 * s, v[s]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (i < left)
                            v[s][i] = widen(y[32 * s + i]);
                }
            }
            float hv[KB][8];
#pragma unroll
            for (int kb = 0; kb < KB; kb++) {
                const int k0 = kBoth ? 8 * (g % 2) : 32 * kb + 8 * g;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    hv[kb][i] = 0.0f;
                if (k0 < p.rank) {
                    const float *h = plan.h + static_cast<int64_t>(row) * R + k0;
                    for (int s = 0; s < p.slices; s++) {
                        float part[8];
                        load8(h + static_cast<int64_t>(s) * p.rows * R, part);
#pragma unroll
                        for (int i = 0; i < 8; i++)
                            hv[kb][i] += part[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; i++)  // past the rank: what padding rows gave
                        hv[kb][i] = k0 + i < p.rank ? hv[kb][i] * scale : 0.0f;
                }
            }
            // f16 has no room for any h: the row's largest is taken to [0.5, 1)
            float unit = 1.0f;
            if constexpr (std::is_same_v<T, _Float16>) {
                float m = 0.0f;
#pragma unroll
                for (int kb = 0; kb < KB; kb++)
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        m = fmaxf(m, fabsf(hv[kb][i]));
                m = fmaxf(m, __shfl_xor(m, 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                const int e = m > 0.0f && m < __builtin_inff() ? min(max(__builtin_amdgcn_frexp_expf(m), -100), 126) : 0;
                unit = ldexpf(1.0f, e);
                const float inv = ldexpf(1.0f, -e);
#pragma unroll
                for (int kb = 0; kb < KB; kb++)
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        hv[kb][i] *= inv;
            }
            f32x4 acc[4] = {};
#pragma unroll
            for (int kb = 0; kb < KB; kb++) {
                Frag<T> hi, lo;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    if constexpr (kSplit) {
                        T a, b;
                        split_value(hv[kb][i], &a, &b);
                        hi.v[i] = kBoth && g >= 2 ? b : a;
                        lo.v[i] = b;
                    } else {
                        hi.v[i] = hv[kb][i];
                    }
                }
#pragma unroll
                for (int f = 0; f < 4; f++) {
                    acc[f] = mma(w[f][kb], hi, acc[f]);
                    if constexpr (kSplit && !kBoth)
                        acc[f] = mma(w[f][kb], lo, acc[f]);
                }
            }
            if (c + r >= t.count)
                continue;
#pragma unroll
            for (int s = 0; s < 2; s++) {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[s][i] += acc[2 * s + i / 4][i % 4] * unit;
                store8(y + 32 * s, p.n - n0 - 32 * s - 8 * g, v[s]);
            }
        }
    }
}

// ---------------------------------------------------------------- host

int padded_rank(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }
int64_t most_tiles(int64_t rows, int64_t adapters, int64_t tile) { return rows / tile + std::min(rows, adapters); }
int64_t whole(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Slices of k: enough workgroups for the chip, none with less than kLeastSlice values.
constexpr int64_t kLeastSlice = 1024, kDownGroups = 256;
void slices_of(int64_t rows, int64_t adapters, int64_t k, int32_t *slices, int32_t *slice) {
    const int64_t tiles = rows <= kSelfRows ? std::min(rows, adapters) : most_tiles(rows, adapters, kDownRows);
    const int64_t s = std::max<int64_t>(1, std::min(kDownGroups / tiles, k / kLeastSlice));
    const int64_t per = std::max<int64_t>(32, ((k + s - 1) / s + 31) / 32 * 32);
    *slice = static_cast<int32_t>(per);
    *slices = static_cast<int32_t>(std::max<int64_t>(1, (k + per - 1) / per));
}

template <typename T, typename SRC, bool SELF>
const void *down_rank(int rank) {
    return rank == 16   ? reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 1, SELF>)
           : rank == 32 ? reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 2, SELF>)
           : rank == 64 ? reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 4, SELF>)
                        : reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 8, SELF>);
}
template <bool SELF>
const void *down_fn(int dtype, int format, int rank) {
    if (format == SSU_FORMAT_MXFP8)
        return down_rank<__bf16, Mx8, SELF>(rank);
    if (format == SSU_FORMAT_MXFP4)
        return down_rank<__bf16, Mx4, SELF>(rank);
    return dtype == SSU_F32   ? down_rank<float, float, SELF>(rank)
           : dtype == SSU_F16 ? down_rank<_Float16, _Float16, SELF>(rank)
                              : down_rank<__bf16, __bf16, SELF>(rank);
}
template <typename T>
const void *up_rank(int rank) {
    return rank == 16   ? reinterpret_cast<const void *>(&lora_up_kernel<T, 16>)
           : rank == 32 ? reinterpret_cast<const void *>(&lora_up_kernel<T, 32>)
           : rank == 64 ? reinterpret_cast<const void *>(&lora_up_kernel<T, 64>)
                        : reinterpret_cast<const void *>(&lora_up_kernel<T, 128>);
}

struct LoraLayout {
    int64_t up, down, perm, h, total;
};
LoraLayout layout(int64_t rows, int64_t adapters, int64_t k, int64_t rank) {
    int32_t slices, slice;
    slices_of(rows, adapters, k, &slices, &slice);
    LoraLayout o;
    o.up = 256;
    o.down = o.up + whole(most_tiles(rows, adapters, kUpRows) * sizeof(Tile));
    o.perm = o.down + whole(most_tiles(rows, adapters, kDownRows) * sizeof(Tile));
    o.h = o.perm + whole(rows * 4);
    o.total = o.h + whole(slices * rows * padded_rank(rank) * 4);
    return o;
}

}  // namespace

int64_t lora_workspace(int64_t rows, int64_t adapters, int64_t k, int64_t rank) { return layout(rows, adapters, k, rank).total; }

int launch_add_lora(const LoraParams &params, int dtype, int format, void *stream) {
    LoraParams p = params;
    slices_of(p.rows, p.adapters, p.k, &p.slices, &p.slice);
    const LoraLayout o = layout(p.rows, p.adapters, p.k, p.rank);
    LoraPlan plan = {reinterpret_cast<int32_t *>(p.workspace), reinterpret_cast<Tile *>(p.workspace + o.up),
                     reinterpret_cast<Tile *>(p.workspace + o.down), reinterpret_cast<int32_t *>(p.workspace + o.perm),
                     reinterpret_cast<float *>(p.workspace + o.h)};
    const int rank = padded_rank(p.rank);
    const unsigned counters = static_cast<unsigned>(p.adapters) * 4;
    void *args[] = {&p, &plan};
    if (p.rows <= kSelfRows) {
        const int64_t groups = 1 + std::min<int64_t>(p.rows, p.adapters) * p.slices;
        if (int hip = launch_groups(down_fn<true>(dtype, format, rank), groups, kDownThreads, args, stream, counters))
            return hip;
    } else {
        if (int hip = launch_groups(reinterpret_cast<const void *>(&lora_plan_kernel), 1, kPlanThreads, args, stream, counters))
            return hip;
        const int64_t groups = most_tiles(p.rows, p.adapters, kDownRows) * p.slices;
        if (int hip = launch_groups(down_fn<false>(dtype, format, rank), groups, kDownThreads, args, stream))
            return hip;
    }
    // workgroups take turns at the items: how many there are is known on the device
    const int64_t blocks = (p.n + kUpWaves * kUpCols - 1) / (kUpWaves * kUpCols);
    const int64_t groups = std::min<int64_t>(most_tiles(p.rows, p.adapters, kUpRows) * blocks, 256 * 8);
    const void *up = dtype == SSU_F32 ? up_rank<float>(rank) : dtype == SSU_F16 ? up_rank<_Float16>(rank) : up_rank<__bf16>(rank);
    return launch_groups(up, groups, kUpThreads, args, stream);
}

}  // namespace ssu
