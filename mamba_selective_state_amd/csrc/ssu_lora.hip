// Low-rank adapters of many requests beside a shared projection (ssu_add_lora):
//   h = x A_i^T (down: k to rank),   y += (scale_i h) B_i^T (up: rank to n),   i the row's adapter.
//
// Rows of one adapter are worked on together, so that each adapter's weights are read once for up to a tile of rows.
// Which rows these are is found on the device: make_plan makes lists of tiles (an adapter and a run of `perm`).
// Up to kSelfRows rows, the down kernel's workgroups look their rows up for themselves, and one more workgroup makes the
// plan for the up kernel in the meantime: two launches. More rows: plan, down, up, and the down kernel's operands go through LDS. 8192 -> 4096:
// 256 rows of 64 adapters take 12.6 us at rank 16 and 49.5 at 128 in two launches, 257 18.0 and 50.5 in three; with one adapter
// 13.5 and 32.3 in two, 16.8 and 26.5 in three.
//
// Bytes bound it, y's above all (read and written): 8192 rows, 4096 -> 18560, rank 64, bf16 8 + 22 + 144 us (608 MB of y at
// 4.2 TB/s), 2048 rows of MXFP8, rank 16, 64 adapters 6 + 7 + 40 (152 MB of y, 46 MB of weights). f32, 2048 rows of rank 128:
// 5 + 45 + 208 us for 12 GFLOP, which f32 matrix instructions do in 76 at best.
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

// A vector's elements moved down by `s` places (not negative), zeros behind them.
template <typename V>
__device__ __forceinline__ V moved_down(V v, int s) {
    if constexpr (sizeof(V) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(V, s < 4 ? b >> (16 * s) : 0);
    } else if constexpr (sizeof(v[0]) == 2) {
        typedef uint64_t U2 __attribute__((ext_vector_type(2)));
        const U2 b = __builtin_bit_cast(U2, v);
        const uint64_t over = b.y << 1 << (63 - 16 * min(s, 3));  // what comes from the upper half, for s < 4
        const U2 r = {s < 4 ? b.x >> (16 * s) | over : s < 8 ? b.y >> (16 * (s - 4)) : 0, s < 4 ? b.y >> (16 * s) : 0};
        return __builtin_bit_cast(V, r);
    } else {
        constexpr int kN = sizeof(V) / 4;
#pragma unroll
        for (int step = 1; step < 2 * kN; step *= 2)
#pragma unroll
            for (int i = 0; i < kN; i++)
                v[i] = !(s & step) ? v[i] : i + step < kN ? v[i + step < kN ? i + step : 0] : 0.0f;
        return s < 2 * kN ? v : V{};
    }
}

// ---------------------------------------------------------------- the plan

constexpr int kDownRows = 32;  // rows of a down tile
constexpr int kUpRows = 128;   // rows of an up tile at most
constexpr int kSelfRows = 256;

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

// By one workgroup of THREADS, PER rows for each thread at a time; `hist`: `adapters` counters in LDS. The order of an adapter's
// rows may differ from call to call; a row's result does not depend on it.
template <int THREADS, int PER>
__device__ void make_plan(const LoraParams &p, const LoraPlan &plan, int *hist) {
    constexpr int kWaves = THREADS / kWaveLanes;
    __shared__ int sums[3][kWaves];
    const int t = threadIdx.x, lane = t % kWaveLanes, wave = t / kWaveLanes;
    int id[PER], number[PER];
    // without branches between them: behind one the compiler waits for each
    auto load_ids = [&](int64_t base) {
        int64_t v[PER];
        if (p.ids_i64) {
#pragma unroll
            for (int u = 0; u < PER; u++)
                v[u] = static_cast<const int64_t *>(p.ids)[min(base + u * THREADS + t, static_cast<int64_t>(p.rows) - 1) * p.ids_s];
        } else {
#pragma unroll
            for (int u = 0; u < PER; u++)
                v[u] = static_cast<const int32_t *>(p.ids)[min(base + u * THREADS + t, static_cast<int64_t>(p.rows) - 1) * p.ids_s];
        }
#pragma unroll
        for (int u = 0; u < PER; u++)
            id[u] = base + u * THREADS + t < p.rows && v[u] >= 0 && v[u] < p.adapters ? static_cast<int>(v[u]) : -1;
    };
    load_ids(0);
    for (int i = t; i < p.adapters; i += THREADS)
        hist[i] = 0;
    __syncthreads();
    constexpr int64_t kBatch = static_cast<int64_t>(THREADS) * PER;
    for (int64_t base = 0;;) {
#pragma unroll
        for (int u = 0; u < PER; u++)
            number[u] = draw_number(hist, id[u], lane);
        base += kBatch;
        if (base >= p.rows)
            break;
        load_ids(base);
    }
    __syncthreads();
    // a run of adapters for each thread: rows, up tiles and down tiles before it
    const int per = (p.adapters + THREADS - 1) / THREADS;
    const int begin = min(t * per, p.adapters), end = min(begin + per, p.adapters);
    int own[3] = {0, 0, 0};
    for (int a = begin; a < end; a++) {
        own[0] += hist[a];
        own[1] += (hist[a] + p.up_rows - 1) / p.up_rows;
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
        for (int i = 0; i < n; i += p.up_rows)
            plan.up[at[1]++] = {a, at[0] + i, min(p.up_rows, n - i), 0};
        for (int i = 0; i < n; i += kDownRows)
            plan.down[at[2]++] = {a, at[0] + i, min(kDownRows, n - i), 0};
        hist[a] = at[0];
        at[0] += n;
    }
    __syncthreads();
    if (p.rows <= kBatch) {  // the first rows' numbers are still known
#pragma unroll
        for (int u = 0; u < PER; u++)
            if (id[u] >= 0)
                plan.perm[hist[id[u]] + number[u]] = u * THREADS + t;
        return;
    }
    for (int64_t base = 0; base < p.rows; base += kBatch) {
        load_ids(base);
#pragma unroll
        for (int u = 0; u < PER; u++) {
            const int to = draw_number(hist, id[u], lane);
            if (id[u] >= 0)
                plan.perm[to] = static_cast<int32_t>(base + u * THREADS + t);
        }
    }
}

constexpr int kPlanThreads = 1024;
__global__ __launch_bounds__(kPlanThreads) void lora_plan_kernel(const LoraParams p, const LoraPlan plan) {
    extern __shared__ int dynamic[];
    make_plan<kPlanThreads, 8>(p, plan, dynamic);
}

// ---------------------------------------------------------------- down

constexpr int kDownThreads = 512;
constexpr int kDownWaves = kDownThreads / kWaveLanes;

// A step is 64 values of k: lane group g's 16 are 16 g .. 16 g + 15, in two operands, of both sides. Four lanes read 128 bytes of
// a row in a row.
template <typename T>
struct Step {
    Frag<T> f[2];
};
template <typename T>
__device__ __forceinline__ Step<T> load_step(const T *p) {
    return {{load_frag(p), load_frag(p + 8)}};
}
template <typename T>
__device__ __forceinline__ Step<T> load_step(const T *p, int n) {
    return {{load_frag(p, n), load_frag(p + 8, n - 8)}};
}

// Rows of x as operands of type T.
template <typename T, typename SRC>
struct XRow {
    const SRC *row;
    __device__ __forceinline__ XRow(const LoraParams &p, int64_t r) : row(static_cast<const SRC *>(p.x) + r * p.x_s) {}
    __device__ __forceinline__ Step<T> load(int at) const { return load_step<T>(row + at); }
    __device__ __forceinline__ Step<T> load(int at, int n) const { return load_step<T>(row + at, n); }
};
// Codes: exact in bf16, which has their four bits and, but for its ends, their scales' range. A lane's 16
// lie in one block of 32.
template <>
struct XRow<__bf16, Mx8> {
    const uint8_t *codes, *scales;
    __device__ __forceinline__ XRow(const LoraParams &p, int64_t r)
        : codes(static_cast<const uint8_t *>(p.x) + r * p.x_s), scales(p.x_scale + r * p.xs_s) {}
    __device__ __forceinline__ Step<__bf16> load(int at) const {
        typedef u32x4 Any4 __attribute__((aligned(1)));
        const u32x4 c = *reinterpret_cast<const Any4 *>(codes + at);
        const uint32_t s = scales[at / 32];
        const float scale = mx8_scale(s);
        Step<__bf16> r;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 lo = e4m3_pair<false>(c[i], scale), hi = e4m3_pair<true>(c[i], scale);
            const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
            for (int j = 0; j < 4; j++)
                r.f[i / 2].v[4 * (i % 2) + j] = narrow<__bf16>(s == 255 ? __builtin_nanf("") : v[j]);
        }
        return r;
    }
    __device__ __forceinline__ Step<__bf16> load(int at, int n) const {
        return n > 0 ? load(at) : Step<__bf16>{{zero_frag<__bf16>(), zero_frag<__bf16>()}};
    }
};
template <>
struct XRow<__bf16, Mx4> {
    const uint8_t *codes, *scales;
    __device__ __forceinline__ XRow(const LoraParams &p, int64_t r)
        : codes(static_cast<const uint8_t *>(p.x) + r * p.x_s), scales(p.x_scale + r * p.xs_s) {}
    __device__ __forceinline__ Step<__bf16> load(int at) const {
        typedef u32x2 Any2 __attribute__((aligned(1)));
        const u32x2 c = *reinterpret_cast<const Any2 *>(codes + at / 2);
        const uint32_t s = scales[at / 32];
        const float scale = mx8_scale(s);
        Step<__bf16> r;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2 v[4] = {e2m1_pair<0>(c[i], scale), e2m1_pair<1>(c[i], scale), e2m1_pair<2>(c[i], scale), e2m1_pair<3>(c[i], scale)};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                r.f[i].v[2 * j] = narrow<__bf16>(s == 255 ? __builtin_nanf("") : v[j].x);
                r.f[i].v[2 * j + 1] = narrow<__bf16>(s == 255 ? __builtin_nanf("") : v[j].y);
            }
        }
        return r;
    }
    __device__ __forceinline__ Step<__bf16> load(int at, int n) const {
        return n > 0 ? load(at) : Step<__bf16>{{zero_frag<__bf16>(), zero_frag<__bf16>()}};
    }
};

// h of up to 16 XF rows of one adapter over values [begin, end) of k. `row_of`(i): the i-th row. Each wave has a run of
// k for itself (in step they would all ask for the same 512 bytes of rows a power of two apart, which the same few channels
// hold), and their sums are joined in LDS, in a fixed order.
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
        Step<T> x[XF], w[RF];
        x[0] = load_x(x0);
        if constexpr (XF > 1)
            x[1] = load_x(x1);
#pragma unroll
        for (int f = 0; f < RF; f++)
            w[f] = load_a(a[f]);
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int i = 0; i < XF; i++)
#pragma unroll
                for (int f = 0; f < RF; f++)
                    acc[i][f] = mma(w[f].f[j], x[i].f[j], acc[i][f]);
    };
    const int per = ((end - begin + kDownWaves - 1) / kDownWaves + 63) / 64 * 64;
    int at = begin + wave * per;
    end = min(end, at + per);
#pragma unroll 2
    for (; at + 64 <= end; at += 64)
        step([&](const XRow<T, SRC> &x) { return x.load(at + 16 * g); }, [&](const T *w) { return load_step(w + at + 16 * g); });
    if (at < end) {
        const int n = end - at - 16 * g;
        step([&](const XRow<T, SRC> &x) { return x.load(at + 16 * g, n); }, [&](const T *w) { return load_step(w + at + 16 * g, n); });
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

// SELF: the workgroups look their rows up for themselves, one pass of up to 16 XF rows of an adapter each, and the first one makes the
// plan. Three waves are enough for eight rows of weights in flight: held to registers for four, 256 rows of 64 adapters, 8192 -> 4096, rank 128, took
// 87.5 us instead of 79.5.
template <typename T, typename SRC, int RF, int XF, bool SELF>
__global__ __launch_bounds__(kDownThreads) __attribute__((amdgpu_waves_per_eu(RF == 8 ? 2 : 1, RF == 8 ? 3 : 8))) void lora_down_kernel(const LoraParams p, const LoraPlan plan) {
    extern __shared__ int dynamic[];
    __shared__ f32x4 sums[kDownWaves * 4 * 64];
    constexpr int kSelfWaves = SELF ? kSelfRows / kWaveLanes : 1;
    static_assert(kSelfRows <= kDownThreads && kSelfRows % kWaveLanes == 0, "a row for each thread");
    __shared__ alignas(16) int rows[SELF ? kSelfRows : 1];
    __shared__ int counts[SELF ? kDownWaves : 1];
    __shared__ int found, found_skip;
    int id = static_cast<int>(blockIdx.x);
    if constexpr (SELF) {
        if (id == 0) {
            make_plan<kDownThreads, 1>(p, plan, dynamic);
            return;
        }
        id--;
    }
    const int slice = id % p.slices;
    const int begin = slice * p.slice, end = min(p.k, begin + p.slice);
    float *h = plan.h + static_cast<int64_t>(slice) * p.rows * (RF * 16);
    if constexpr (SELF) {
        constexpr int kPass = 16 * XF;
        const int t = threadIdx.x, lane = t % kWaveLanes, wave = __builtin_amdgcn_readfirstlane(t / kWaveLanes);
        const int group = id / p.slices, heads = min(p.rows, p.adapters) * p.parts;
        // thread t has row t
        const int id_here = t < p.rows ? adapter_of(p, t) : -1;
        // The pass: from the `skip`-th of the adapter's rows on.
        int adapter = group / p.parts, skip = group % p.parts * kPass, from = -1;
        if (group >= heads) {
            // the passes that are left, in the adapters' order
            for (int i = t; i < p.adapters; i += kDownThreads)
                dynamic[i] = 0;
            if (t == 0)
                found = -1;
            __syncthreads();
            draw_number(dynamic, id_here, lane);
            __syncthreads();
            auto passes = [&](int i) { return max(0, (dynamic[i] + kPass - 1) / kPass - p.parts); };
            const int per = (p.adapters + kDownThreads - 1) / kDownThreads;
            const int first = min(t * per, p.adapters), last = min(first + per, p.adapters);
            int own = 0;
            for (int i = first; i < last; i++)
                own += passes(i);
            int at = own;
#pragma unroll
            for (int d = 1; d < kWaveLanes; d *= 2) {
                const int o = __shfl_up(at, d);
                at += lane >= d ? o : 0;
            }
            if (lane == kWaveLanes - 1)
                counts[wave] = at;
            at -= own;
            __syncthreads();
            for (int w = 0; w < wave; w++)
                at += counts[w];
            int left = group - heads - at;
            if (left >= 0 && left < own) {
                int i = first;
                for (; left >= passes(i); i++)
                    left -= passes(i);
                found = i;
                found_skip = (p.parts + left) * kPass;
            }
            __syncthreads();
            adapter = __builtin_amdgcn_readfirstlane(found), skip = __builtin_amdgcn_readfirstlane(found_skip);
            if (adapter < 0)
                return;
        } else if (p.rows < p.adapters) {
            from = group;
            adapter = __builtin_amdgcn_readfirstlane(adapter_of(p, from));
            if (adapter < 0)
                return;
        }
        // the adapter's rows in their own order, the same for every pass
        const uint64_t which = __ballot(id_here == adapter);
        if (lane == 0)
            counts[wave] = __popcll(which);
        __syncthreads();
        int at = __popcll(which & ((1ull << lane) - 1)), n = 0;
#pragma unroll
        for (int w = 0; w < kSelfWaves; w++) {
            at += w < wave ? counts[w] : 0;
            n += counts[w];
        }
        n = __builtin_amdgcn_readfirstlane(n);
        if (id_here == adapter)
            rows[at] = t;
        if (t == from)
            found_skip = at;
        __syncthreads();
        if (from >= 0) {
            skip = __builtin_amdgcn_readfirstlane(found_skip);
            if (skip % kPass != 0)
                return;
        }
        if (skip < n)
            down_tile<T, SRC, RF, XF>(p, adapter, min(kPass, n - skip), begin, end, h, sums, [&](int j) { return rows[skip + j]; });
    } else {
        const int tile = id / p.slices;
        if (tile >= plan.counts[1])
            return;
        const Tile t = plan.down[tile];
        down_tile<T, SRC, RF, XF>(p, t.adapter, t.count, begin, end, h, sums, [&](int j) { return plan.perm[t.first + j]; });
    }
}

// ---------------------------------------------------------------- down, many rows
//
// Tiles of the plan, through LDS: a stage is 256 bytes (128 or, in f32, 64 values of k) of 32 rows of x and of all rank rows, which
// LDS-DMA brings in whole lines, two stages ahead. 8192 x 4096 bf16 of rank 64 take 22 us (67 MB of x, part of it from the last-level cache, and A once for each 32 rows, 134 MB
// from the L2s), 35 with x from HBM; with operands straight from memory, 64 bytes of 16 rows for each access, 50.
//
// Chunk c (16 bytes) of row r is at place c ^ r of its row, so that the 16 rows of an operand are read from different banks.

constexpr int kStageBytes = 256;  // of a row of T

// x's part of a stage: bytes of a row, and how an operand is read from them.
template <typename T, typename SRC>
struct XStage {
    static constexpr int kRow = kStageBytes;
    // `at`: the row's image; chunks' places are swapped by `swap`
    static __device__ __forceinline__ Frag<T> read(const uint8_t *at, int swap, int step, int g, uint32_t) {
        Frag<T> f;
        if constexpr (sizeof(T) == 2) {
            f = *reinterpret_cast<const Frag<T> *>(at + ((4 * step + g) ^ swap) * 16);
        } else {
            *reinterpret_cast<f32x4 *>(&f.v) = *reinterpret_cast<const f32x4 *>(at + ((8 * step + 2 * g) ^ swap) * 16);
            *(reinterpret_cast<f32x4 *>(&f.v) + 1) = *reinterpret_cast<const f32x4 *>(at + ((8 * step + 2 * g + 1) ^ swap) * 16);
        }
        return f;
    }
};
template <>
struct XStage<__bf16, Mx8> {
    static constexpr int kRow = kStageBytes / 2;
    static __device__ __forceinline__ Frag<__bf16> read(const uint8_t *at, int swap, int step, int g, uint32_t scales) {
        const u32x2 c = *reinterpret_cast<const u32x2 *>(at + ((2 * step + g / 2) ^ (swap / 2 % 8)) * 16 + g % 2 * 8);
        const uint32_t s = (scales >> (8 * step)) & 0xFF;
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
};
template <>
struct XStage<__bf16, Mx4> {
    static constexpr int kRow = kStageBytes / 4;
    static __device__ __forceinline__ Frag<__bf16> read(const uint8_t *at, int swap, int step, int g, uint32_t scales) {
        const uint32_t c = *reinterpret_cast<const uint32_t *>(at + (step ^ (swap / 4 % 4)) * 16 + g * 4);
        const uint32_t s = (scales >> (8 * step)) & 0xFF;
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
};

template <typename T, typename SRC, int RF>
__global__ __launch_bounds__(kDownThreads) void lora_down_staged_kernel(const LoraParams p, const LoraPlan plan) {
    constexpr bool kCodes = std::is_same_v<SRC, Mx8> || std::is_same_v<SRC, Mx4>;
    using Stage = XStage<T, SRC>;
    constexpr int kDepth = kStageBytes / static_cast<int>(sizeof(T)), kSteps = kDepth / 32;
    constexpr int kXRow = Stage::kRow, kXBytes = kDownRows * kXRow, kABytes = RF * 16 * kStageBytes, kBytes = kXBytes + kABytes;
    // KiB of a stage, and for codes the rows' scale words; of a wave, and how many waves have one more
    constexpr int kWhole = kBytes / 1024, kFills = kWhole + kCodes, kEach = kFills / kDownWaves, kMore = kFills % kDownWaves;
    constexpr int kScaleBytes = kCodes ? 256 : 0;
    constexpr int kRing = RF == 8 ? 2 : 3;
    constexpr int kPairs = kDownRows / 16 * RF;  // of an operand of x and one of A
    constexpr int kMine = kPairs > kDownWaves ? kPairs / kDownWaves : 1;
    constexpr int kSubs = kPairs >= kDownWaves ? 1 : kDownWaves / kPairs < kSteps ? kDownWaves / kPairs : kSteps;  // waves of a pair: turns at the steps
    // arrays of their own: the compiler tells fills of one from reads of another
    __shared__ alignas(16) uint8_t s0[kBytes + kScaleBytes], s1[kBytes + kScaleBytes], s2[kRing > 2 ? kBytes + kScaleBytes : 16];
    __shared__ f32x4 sums[kSubs > 1 ? kDownWaves * 64 : 1];
    const int tile = static_cast<int>(blockIdx.x) / p.slices, slice = static_cast<int>(blockIdx.x) % p.slices;
    if (tile >= plan.counts[1])
        return;
    const Tile t = plan.down[tile];
    const int lane = threadIdx.x % kWaveLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int r = lane % 16, g = lane / 16;
    const int begin = slice * p.slice, end = min(p.k, begin + p.slice), stages = (end - begin) / kDepth;
    constexpr int64_t kUnit = static_cast<int64_t>(sizeof(T));
    const uint8_t *a = static_cast<const uint8_t *>(p.a) + t.adapter * p.a_l * kUnit;
    // what this wave fills: KiB number wave + 8 i of a stage, x's first
    const uint8_t *src[kEach + 1];
    int advance[kEach + 1];
#pragma unroll
    for (int i = 0; i <= kEach; i++) {
        const int fill = wave + i * kDownWaves;
        if (fill < kXBytes / 1024) {
            constexpr int kLanes = kXRow / 16;
            const int row = fill * (1024 / kXRow) + lane / kLanes, slot = lane % kLanes;
            const int swap = kXRow == 256 ? row % 16 : kXRow == 128 ? row % 16 / 2 : row % 16 / 4;
            const int64_t stride = kCodes ? p.x_s : p.x_s * kUnit;
            src[i] = static_cast<const uint8_t *>(p.x) + plan.perm[t.first + min(row, t.count - 1)] * stride +
                     static_cast<int64_t>(begin / kDepth) * kXRow + (slot ^ swap) * 16;
            advance[i] = kXRow;
        } else if (kCodes && fill >= kWhole) {
            src[i] = p.x_scale + plan.perm[t.first + min(lane % kDownRows, t.count - 1)] * p.xs_s + begin / 32;
            advance[i] = kSteps;
        } else {
            const int row = (fill - kXBytes / 1024) * 4 + lane / 16, slot = lane % 16;
            src[i] = a + min(row, p.rank - 1) * p.a_r * kUnit + begin * kUnit + (slot ^ (row % 16)) * 16;
            advance[i] = kStageBytes;
        }
    }
    // the waits count fetches in the order in which they are written down here
    auto in_order = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto fill = [&](int stage, uint8_t *image) {
        in_order();
#pragma unroll
        for (int i = 0; i <= kEach; i++) {
            if (i == kEach && wave >= kMore)
                break;
            const int fill = wave + i * kDownWaves;
            const auto *from = (const __attribute__((address_space(1))) void *)(src[i] + static_cast<int64_t>(stage) * advance[i]);
            auto *to = (__attribute__((address_space(3))) void *)(image + fill * 1024);
            if (kCodes && i == kFills / kDownWaves - (kFills % kDownWaves == 0) && fill == kWhole)
                __builtin_amdgcn_global_load_lds(from, to, 4, 0, 0);
            else
                __builtin_amdgcn_global_load_lds(from, to, 16, 0, 0);
        }
        in_order();
    };
    // Barrier behind which the next stage's fills, all but `left` of this wave's, have arrived, and the last
    // stage's image has been read. Spelled out: a barrier with the compiler's own waits would wait for all fills.
    auto meet = [&](auto left) {
        in_order();
        __builtin_amdgcn_s_waitcnt(0x0070 | decltype(left)::value);  // vmcnt(left) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        in_order();
    };
    const int pair0 = kPairs >= kDownWaves ? wave * kMine : wave % kPairs, sub = kPairs >= kDownWaves ? 0 : wave / kPairs;
    const int xf = pair0 / RF;  // pairs of a wave share x's operand
    const int x_row = plan.perm[t.first + min(16 * xf + r, t.count - 1)];
    f32x4 acc[kMine] = {};
    auto image = [&](int i) { return i == 0 ? s0 : i == 1 ? s1 : s2; };
    for_passes<0, kRing - 1>([&](auto i) {
        if (decltype(i)::value < stages)
            fill(decltype(i)::value, image(decltype(i)::value));
    });
    for (int first = 0; first < stages; first += kRing)
        for_passes<0, kRing>([&](auto i) {
            constexpr int n = decltype(i)::value;
            const int stage = first + n;
            if (stage >= stages)
                return;
            // the next stage's fills may still be on their way
            if (kRing == 2 || stage + 1 >= stages)
                meet(std::integral_constant<int, 0>());
            else if (wave < kMore)
                meet(std::integral_constant<int, kEach + 1>());
            else
                meet(std::integral_constant<int, kEach>());
            if (stage + kRing - 1 < stages)
                fill(stage + kRing - 1, image((n + kRing - 1) % kRing));
            const uint8_t *x_image = image(n) + (16 * xf + r) * kXRow, *a_image = image(n) + kXBytes;
            const uint32_t scales = kCodes ? *reinterpret_cast<const uint32_t *>(image(n) + kBytes + (16 * xf + r) * 4) : 0;
#pragma unroll
            for (int step = 0; step < kSteps; step++) {
                if (kSubs > 1 && step % kSubs != sub)
                    continue;
                const Frag<T> x = Stage::read(x_image, r, step, g, scales);
#pragma unroll
                for (int m = 0; m < kMine; m++) {
                    const Frag<T> w = XStage<T, T>::read(a_image + ((pair0 + m) % RF * 16 + r) * kStageBytes, r, step, g, 0);
                    acc[m] = mma(w, x, acc[m]);
                }
            }
        });
    // what is left of k, straight from memory
    for (int at = begin + stages * kDepth + 32 * sub; at < end && sub < kSubs; at += 32 * kSubs) {
        const int n = end - at - 8 * g;
        Frag<T> x;
        if constexpr (kCodes) {
            x = zero_frag<T>();
            if (n > 0) {  // a lane's eight of the sixteen that the other kernel takes
                const Step<T> both = XRow<T, SRC>(p, x_row).load(at + g / 2 * 16);
                x.v = g % 2 ? both.f[1].v : both.f[0].v;
            }
        } else {
            x = load_frag(static_cast<const T *>(p.x) + x_row * p.x_s + at + 8 * g, n);
        }
#pragma unroll
        for (int m = 0; m < kMine; m++) {
            const T *row = reinterpret_cast<const T *>(a) + min((pair0 + m) % RF * 16 + r, p.rank - 1) * p.a_r;
            acc[m] = mma(load_frag(row + at + 8 * g, n), x, acc[m]);
        }
    }
    if constexpr (kSubs > 1) {
        sums[wave * 64 + lane] = acc[0];
        __syncthreads();
        if (sub != 0)
            return;
#pragma unroll
        for (int i = 1; i < kSubs; i++)
            acc[0] += sums[(wave + i * kPairs) * 64 + lane];
    }
    if (sub == 0 && 16 * xf + r < t.count) {
        float *h = plan.h + (static_cast<int64_t>(slice) * p.rows + x_row) * (RF * 16) + 4 * g;
#pragma unroll
        for (int m = 0; m < kMine; m++)
            *reinterpret_cast<f32x4 *>(h + (pair0 + m) % RF * 16) = acc[m];
    }
}

// ---------------------------------------------------------------- up

constexpr int kUpThreads = 256;
constexpr int kUpWaves = kUpThreads / kWaveLanes;
constexpr int kUpCols = 64;  // of a wave

// A value as two summands of T, the first of the value's sign: in f16 what is too small for one is the smallest less itself.
template <typename T>
__device__ __forceinline__ void split_value(float v, T *hi, T *lo) {
    *hi = narrow<T>(v);
    if constexpr (std::is_same_v<T, _Float16>)
        *hi = *hi == static_cast<T>(0.0f) && v != 0.0f ? static_cast<T>(copysignf(0x1p-24f, v)) : *hi;
    const float w = widen(*hi);
    *lo = narrow<T>(fabsf(w) < __builtin_inff() ? v - w : 0.0f);
}

// A tile of rows times four waves' columns. Every wave fetches its columns' weights row by row and takes them to
// registers through LDS; h of the tile is joined over the slices of k, scaled, split and left in LDS; then the waves go through the
// rows, 16 at a time.
//
// Here h's rows go first and the weights second: lane l has results of rows 4 (l / 16) .. + 3, and fragment f's column l % 16 is
// output 4 (l % 16) + f of the wave's, so that 16 lanes in a row have 64 outputs in a row of one row of y. With rows in the lanes, 16
// lines for every 16 lanes, 8192 x 18560 bf16 of rank 64 took 200 us instead of 138.
//
// PAST: y goes past the caches both ways, which keep x and the weights: 8192 x 18560 of rank 64 with the first product 184
// us, so 174 (with the writes alone 184). Rows that share lines (an odd number of outputs) need the caches: 777 x 2049
// f16 18.6 us, past them 20.0.
template <typename T, int R, bool PAST>
__global__ __launch_bounds__(kUpThreads, sizeof(T) == 2 && R <= 64 ? 4 : 2) void lora_up_kernel(const LoraParams p, const LoraPlan plan) {
    constexpr int N = 4;                     // outputs of a lane and row
    constexpr int KB = R < 32 ? 1 : R / 32;  // operands of 32 along the rank
    constexpr bool kSplit = sizeof(T) == 2;
    constexpr bool kBoth = kSplit && R == 16;                    // hi and lo fill one operand
    constexpr int kHRow = R * 4 + 16;                            // bytes of a row of h in LDS: no two of 16 rows start in the same bank
    constexpr int kBRow = R * static_cast<int>(sizeof(T)) + 16;  // and of the weights
    constexpr int kPieces = R / 8;                               // of eight values, of a row; as many for each lane
    constexpr int kHRows = kUpThreads / (R / 4);                 // rows of h at a time
    // a chunk of y ahead, where the registers leave room for it and four waves: 8192 x 18560 bf16 of rank 64 take 132 us without
    // it and 145 with it and three waves, 2048 x 18560 of rank 16 48 and 42
    constexpr bool kAhead = R <= 32;
    constexpr bool kScaled = std::is_same_v<T, _Float16>;
    // lo times an infinite weight is NaN where lo is 0, and an infinity of lo's sign otherwise; hi has h's sign. Products beyond f32's range
    // are the same. So where a sum is NaN, it is that of hi alone. A look at every sum took 2048 x 18560 of rank 16 from 53.4 to 57
    // us; there, where hi and lo have weights of their own, lo's are 0 for infinite ones (in bf16 from 2^64 on: 8 bits of h are left for them),
    // and bf16 rows of an h of 2^64 or more are taken by 2^-100 through the products: 54.1 us.
    constexpr bool kLook = kSplit && !kBoth, kLess = kBoth && !kScaled;
    constexpr float kLarge = kScaled ? __builtin_inff() : 0x1p64f;
    typedef T Y __attribute__((ext_vector_type(N)));
    typedef T AnyY __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    typedef int64_t L2 __attribute__((ext_vector_type(2)));
    __shared__ alignas(16) uint8_t staged[std::max(kUpRows * kHRow, kUpWaves * kUpCols * kBRow)];
    __shared__ alignas(16) int64_t y_rows[kUpRows];  // where the rows are in y
    __shared__ int32_t rows[kUpRows];
    __shared__ alignas(16) float units[kScaled || kLess ? kUpRows : 4];  // what the rows' sums are multiplied by
    const int lane = threadIdx.x % kWaveLanes, wave = threadIdx.x / kWaveLanes;
    const int r = lane % 16, g = lane / 16;
    uint8_t *b_rows = staged + wave * kUpCols * kBRow, *h_rows = staged;
    const uint32_t blocks = (p.n + kUpWaves * kUpCols - 1) / (kUpWaves * kUpCols);
    const uint32_t items = static_cast<uint32_t>(plan.counts[0]) * blocks;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const Tile t = plan.up[item / blocks];
        const int col0 = (static_cast<int>(item % blocks) * kUpWaves + wave) * kUpCols;
        const int left = p.n - col0 - N * r;  // of the lane's outputs
        const bool whole = col0 + kUpCols <= p.n;  // the wave's outputs all exist
        // what is needed first is asked for at once: the tile's rows, weights, then the rows' first h and y
        const int row_lo = plan.perm[t.first + min(lane, t.count - 1)];
        const int part = threadIdx.x % (R / 4) * 4, h_first = threadIdx.x / (R / 4);
        const T *b = static_cast<const T *>(p.b) + t.adapter * p.b_l;
        Frag<T> piece[kPieces];
        if (p.rank == R) {
#pragma unroll
            for (int u = 0; u < kPieces; u++) {
                const int q = u * kWaveLanes + lane;
                piece[u] = load_frag(b + min(col0 + q / kPieces, p.n - 1) * p.b_n + q % kPieces * 8);
            }
        } else {
#pragma unroll
            for (int u = 0; u < kPieces; u++) {
                // a row's last eight values hold its end; what lies past it becomes 0
                const int q = u * kWaveLanes + lane, c = q % kPieces * 8, from = max(0, min(c, p.rank - 8));
                const T *row = b + min(col0 + q / kPieces, p.n - 1) * p.b_n;
                if (p.rank >= 8) {
                    piece[u].v = moved_down(load_frag(row + from).v, c - from);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const T value = row[min(i, p.rank - 1)];
                        piece[u].v[i] = c + i < p.rank ? value : static_cast<T>(0.0f);
                    }
                }
            }
        }
        auto h_at = [&](int row) {
            const float *src = plan.h + static_cast<int64_t>(row) * R + part;
            f32x4 v = *reinterpret_cast<const f32x4 *>(src);
            for (int s = 1; s < p.slices; s++)
                v += *reinterpret_cast<const f32x4 *>(src + s * static_cast<int64_t>(p.rows) * R);
            return v;
        };
        const f32x4 h0 = h_at(__shfl(row_lo, h_first));
        T *y = static_cast<T *>(p.y) + col0 + N * r;
        Y v[4];  // a chunk's outputs, as they are until they are used
        auto read_y = [](const T *at) -> Y {
            const AnyY *y = reinterpret_cast<const AnyY *>(at);
            return PAST ? __builtin_nontemporal_load(y) : *y;
        };
        auto write_y = [](T *at, const Y &value) {
            AnyY *y = reinterpret_cast<AnyY *>(at);
            if constexpr (PAST)
                __builtin_nontemporal_store(static_cast<AnyY>(value), y);
            else
                *y = value;
        };
        T *to[4];
        if (kAhead && whole) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                to[i] = y + __shfl(row_lo, 4 * g + i) * p.y_s;
                v[i] = read_y(to[i]);
            }
        }
        __syncthreads();  // the last item's h and rows have been read
        if (threadIdx.x < kUpRows) {
            const int row = plan.perm[t.first + min(static_cast<int>(threadIdx.x), t.count - 1)];
            rows[threadIdx.x] = row;
            y_rows[threadIdx.x] = row * p.y_s;
        }
#pragma unroll
        for (int u = 0; u < kPieces; u++) {
            const int q = u * kWaveLanes + lane;
            *reinterpret_cast<Frag<T> *>(b_rows + q / kPieces * kBRow + q % kPieces * 8 * static_cast<int>(sizeof(T))) = piece[u];
        }
        bool past = false;  // whether a weight of the wave's is large
        if constexpr (kBoth) {
            typedef uint16_t U2 __attribute__((ext_vector_type(2)));
            U2 most = {0, 0};
#pragma unroll
            for (int u = 0; u < kPieces; u++) {
                const u32x4 bits = __builtin_bit_cast(u32x4, piece[u].v);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    most = __builtin_elementwise_max(most, __builtin_bit_cast(U2, bits[i] & 0x7FFF7FFFu));
            }
            past = __ballot(max(most.x, most.y) >= __builtin_bit_cast(uint16_t, static_cast<T>(kLarge))) != 0;
        }
        wave_lds_fence();
        Frag<T> w[N][KB];
#pragma unroll
        for (int f = 0; f < N; f++)
#pragma unroll
            for (int kb = 0; kb < KB; kb++) {
                const int k0 = kBoth ? 8 * (g % 2) : 32 * kb + 8 * g;
                if (k0 < R)
                    w[f][kb] = *reinterpret_cast<const Frag<T> *>(b_rows + (N * r + f) * kBRow + k0 * static_cast<int>(sizeof(T)));
                else
                    w[f][kb] = zero_frag<T>();
            }
        if (kBoth && past) {
#pragma unroll
            for (int f = 0; f < N; f++)
#pragma unroll
                for (int i = 0; i < 8; i++)
                    w[f][0].v[i] = g < 2 || fabsf(widen(w[f][0].v[i])) < kLarge ? w[f][0].v[i] : static_cast<T>(0.0f);
        }
        __syncthreads();
        // h, 16 bytes of a row for each lane, whole lines by lanes in a row
        const float scale = p.scale ? p.scale[t.adapter * p.scale_s] : 1.0f;
        for (int row = h_first; row < (t.count + kHRows - 1) / kHRows * kHRows; row += kHRows) {
            f32x4 v = row == h_first ? h0 : h_at(rows[row]);
#pragma unroll
            for (int j = 0; j < 4; j++)  // past the rank: what padding rows gave
                v[j] = part + j < p.rank ? v[j] * scale : 0.0f;
            float inv = 1.0f;
            if constexpr (kScaled) {
                // f16 has no room for any h: the row's largest finite one is taken to [0.5, 1)
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; j++)
                    m = fmaxf(m, fabsf(v[j]) < __builtin_inff() ? fabsf(v[j]) : 0.0f);
#pragma unroll
                for (int d = 1; d < R / 4; d *= 2)
                    m = fmaxf(m, __shfl_xor(m, d));
                const int e = m > 0.0f ? min(max(__builtin_amdgcn_frexp_expf(m), -100), 126) : 0;
                inv = ldexpf(1.0f, -e);
                units[row] = ldexpf(1.0f, e);
            }
            if constexpr (kLess) {
                float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))), unit = 1.0f;
                if (__ballot(m >= kLarge)) {
#pragma unroll
                    for (int d = 1; d < R / 4; d *= 2)
                        m = fmaxf(m, __shfl_xor(m, d));
                    inv = m >= kLarge ? 0x1p-100f : 1.0f;
                    unit = m >= kLarge ? 0x1p100f : 1.0f;
                }
                units[row] = unit;
            }
            uint8_t *dst = h_rows + row * kHRow;
            if constexpr (kSplit) {
                typedef T V4 __attribute__((ext_vector_type(4)));
                V4 hi, lo;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    T a, b;
                    split_value(v[j] * inv, &a, &b);
                    hi[j] = a;
                    lo[j] = b;
                }
                *reinterpret_cast<V4 *>(dst + part * 2) = hi;
                *reinterpret_cast<V4 *>(dst + (R + part) * 2) = lo;
            } else {
                *reinterpret_cast<f32x4 *>(dst + part * 4) = v;
            }
        }
        __syncthreads();
        // v += delta, for the chunk from row c on
        auto add = [&](int c) {
            const uint8_t *h = h_rows + (c + r) * kHRow;
            f32x4 acc[N] = {};
#pragma unroll
            for (int kb = 0; kb < KB; kb++) {
                if constexpr (kBoth) {
                    const Frag<T> b = load_frag(reinterpret_cast<const T *>(h + 16 * g));
#pragma unroll
                    for (int f = 0; f < N; f++)
                        acc[f] = mma(b, w[f][kb], acc[f]);
                } else if constexpr (kSplit) {
                    const Frag<T> hi = load_frag(reinterpret_cast<const T *>(h + 64 * kb + 16 * g));
                    const Frag<T> lo = load_frag(reinterpret_cast<const T *>(h + 2 * R + 64 * kb + 16 * g));
#pragma unroll
                    for (int f = 0; f < N; f++)
                        acc[f] = mma(hi, w[f][kb], acc[f]);
#pragma unroll
                    for (int f = 0; f < N; f++)
                        acc[f] = mma(lo, w[f][kb], acc[f]);
                } else {
                    const Frag<T> b = R >= 32 || g < 2 ? load_frag(reinterpret_cast<const T *>(h + 128 * kb + 32 * g)) : zero_frag<T>();
#pragma unroll
                    for (int f = 0; f < N; f++)
                        acc[f] = mma(b, w[f][kb], acc[f]);
                }
            }
            if constexpr (kLook) {
                bool nan = false;
#pragma unroll
                for (int f = 0; f < N; f++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        nan = nan || acc[f][i] != acc[f][i];
                if (__ballot(nan)) {
#pragma unroll
                    for (int f = 0; f < N; f++) {
                        __builtin_amdgcn_sched_barrier(0);  // one at a time: few registers
                        f32x4 alone = {};
#pragma unroll
                        for (int kb = 0; kb < KB; kb++)
                            alone = mma(load_frag(reinterpret_cast<const T *>(h + 64 * kb + 16 * g)), w[f][kb], alone);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            acc[f][i] = acc[f][i] != acc[f][i] ? alone[i] : acc[f][i];
                    }
                }
            }
            f32x4 unit = {1.0f, 1.0f, 1.0f, 1.0f};
            if constexpr (kScaled || kLess)
                unit = *reinterpret_cast<const f32x4 *>(units + c + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int f = 0; f < N; f++)
                    v[i][f] = narrow<T>(widen(v[i][f]) + acc[f][i] * unit[i]);
        };
        auto places = [&](int c, T *(&to)[4]) {
            const L2 *at = reinterpret_cast<const L2 *>(y_rows + c + 4 * g);
            to[0] = y + at[0].x, to[1] = y + at[0].y, to[2] = y + at[1].x, to[3] = y + at[1].y;
        };
        auto load = [&](int c) {
            places(c, to);
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[i] = read_y(to[i]);
        };
        int c = 0;
        if (whole) {
#pragma unroll 1
            for (; c + 16 <= t.count; c += 16) {
                if constexpr (kAhead) {
                    // the next chunk is on its way while one is worked on; no store is waited for
                    T *next_to[4];
                    Y next[4];
                    if (c + 16 < t.count) {
                        places(c + 16, next_to);
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            next[i] = read_y(next_to[i]);
                    }
                    add(c);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        write_y(to[i], v[i]);
                        to[i] = next_to[i];
                        v[i] = next[i];
                    }
                } else {
                    load(c);
                    add(c);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        write_y(to[i], v[i]);
                }
            }
            if (c < t.count) {
                if constexpr (!kAhead)
                    load(c);
                add(c);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (c + 4 * g + i < t.count)
                        write_y(to[i], v[i]);
            }
        } else {
            const int past = max(0, N - left);  // how far the lane's outputs reach past the row's end
#pragma unroll 1
            for (; c < t.count; c += 16) {
                places(c, to);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (p.n >= N) {
                        v[i] = moved_down(static_cast<Y>(*reinterpret_cast<const AnyY *>(to[i] - past)), past);
                    } else {
#pragma unroll
                        for (int f = 0; f < N; f++)
                            v[i][f] = to[i][min(f, left - 1)];
                    }
                }
                add(c);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (c + 4 * g + i < t.count)
#pragma unroll
                        for (int f = 0; f < N; f++)
                            if (f < left)
                                to[i][f] = v[i][f];
            }
        }
    }
}

// ---------------------------------------------------------------- host

int padded_rank(int64_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }
int64_t most_tiles(int64_t rows, int64_t adapters, int64_t tile) { return rows / tile + std::min(rows, adapters); }
int64_t whole(int64_t bytes) { return (bytes + 255) / 256 * 256; }

constexpr int64_t kUpGroups = 8192;  // some times what the chip holds at once
// Slices of k: enough workgroups for the chip, none with less than kLeastSlice values. Every item of the second product adds the
// slices up: 256 rows of 64 adapters, 8192 -> 4096, take 7.3 + 5.8 us with four slices and 7.0 + 6.8 with eight. How many of the adapters have
// rows is not known here; the rule takes all that can. 512 rows of rank 128 with 512 adapters in the table: 193 us where 300 have rows, 62 where one
// has; with no more than 64 of them counted 228 and 30. Rank 16: 43 and 27, 45 and 18.
constexpr int64_t kLeastSlice = 512, kSelfGroups = 256, kDownGroups = 512, kMostSlices = 4;
constexpr int64_t kMostParts = 8;
void slices_of(int64_t rows, int64_t adapters, int64_t k, int32_t *slices, int32_t *slice) {
    const int64_t tiles = rows <= kSelfRows ? std::min(rows, adapters) : most_tiles(rows, adapters, kDownRows);
    const int64_t groups = rows <= kSelfRows ? kSelfGroups : kDownGroups;
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>({(groups + tiles - 1) / tiles, k / kLeastSlice, kMostSlices}));
    const int64_t per = std::max<int64_t>(128, ((k + s - 1) / s + 127) / 128 * 128);  // whole stages
    *slice = static_cast<int32_t>(per);
    *slices = static_cast<int32_t>(std::max<int64_t>(1, (k + per - 1) / per));
}

template <typename T, typename SRC, int XF, bool SELF>
const void *down_rank(int rank) {
    return rank == 16   ? reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 1, XF, SELF>)
           : rank == 32 ? reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 2, XF, SELF>)
           : rank == 64 ? reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 4, XF, SELF>)
                        : reinterpret_cast<const void *>(&lora_down_kernel<T, SRC, 8, XF, SELF>);
}
template <int XF, bool SELF>
const void *down_fn(int dtype, int format, int rank) {
    if (format == SSU_FORMAT_MXFP8)
        return down_rank<__bf16, Mx8, XF, SELF>(rank);
    if (format == SSU_FORMAT_MXFP4)
        return down_rank<__bf16, Mx4, XF, SELF>(rank);
    return dtype == SSU_F32   ? down_rank<float, float, XF, SELF>(rank)
           : dtype == SSU_F16 ? down_rank<_Float16, _Float16, XF, SELF>(rank)
                              : down_rank<__bf16, __bf16, XF, SELF>(rank);
}
template <typename T, typename SRC>
const void *staged_rank(int rank) {
    return rank == 16   ? reinterpret_cast<const void *>(&lora_down_staged_kernel<T, SRC, 1>)
           : rank == 32 ? reinterpret_cast<const void *>(&lora_down_staged_kernel<T, SRC, 2>)
           : rank == 64 ? reinterpret_cast<const void *>(&lora_down_staged_kernel<T, SRC, 4>)
                        : reinterpret_cast<const void *>(&lora_down_staged_kernel<T, SRC, 8>);
}
const void *staged_fn(int dtype, int format, int rank) {
    if (format == SSU_FORMAT_MXFP8)
        return staged_rank<__bf16, Mx8>(rank);
    if (format == SSU_FORMAT_MXFP4)
        return staged_rank<__bf16, Mx4>(rank);
    return dtype == SSU_F32   ? staged_rank<float, float>(rank)
           : dtype == SSU_F16 ? staged_rank<_Float16, _Float16>(rank)
                              : staged_rank<__bf16, __bf16>(rank);
}
// Whether LDS-DMA can fetch x and a, 16 bytes from places that are multiples of them, and words of scales.
bool staged_fits(const LoraParams &p, int dtype, int format) {
    const int64_t unit = dtype == SSU_F32 ? 4 : 2, x_unit = format == SSU_FORMAT_SAME ? unit : 1;
    auto whole16 = [](const void *at) { return reinterpret_cast<uintptr_t>(at) % 16 == 0; };
    if (format != SSU_FORMAT_SAME && (reinterpret_cast<uintptr_t>(p.x_scale) % 4 != 0 || p.xs_s % 4 != 0))
        return false;
    return whole16(p.x) && whole16(p.a) && p.x_s * x_unit % 16 == 0 && p.a_l * unit % 16 == 0 && p.a_r * unit % 16 == 0;
}
template <typename T, bool PAST>
const void *up_rank(int rank) {
    return rank == 16   ? reinterpret_cast<const void *>(&lora_up_kernel<T, 16, PAST>)
           : rank == 32 ? reinterpret_cast<const void *>(&lora_up_kernel<T, 32, PAST>)
           : rank == 64 ? reinterpret_cast<const void *>(&lora_up_kernel<T, 64, PAST>)
                        : reinterpret_cast<const void *>(&lora_up_kernel<T, 128, PAST>);
}
template <bool PAST>
const void *up_fn(int dtype, int rank) {
    return dtype == SSU_F32 ? up_rank<float, PAST>(rank) : dtype == SSU_F16 ? up_rank<_Float16, PAST>(rank) : up_rank<__bf16, PAST>(rank);
}
// Whether y's rows begin at whole lines.
bool whole_lines(const LoraParams &p, int dtype) {
    return reinterpret_cast<uintptr_t>(p.y) % 128 == 0 && p.y_s * (dtype == SSU_F32 ? 4 : 2) % 128 == 0;
}

// Rows of an up tile: shorter ones where there would be too few items for the chip (622 rows of 11 adapters, 2049 outputs: 8.4 us, with
// 128 rows 12).
constexpr int64_t kFewItems = 1024;
int up_rows_of(int64_t rows, int64_t n) {
    const int64_t blocks = (n + kUpWaves * kUpCols - 1) / (kUpWaves * kUpCols);
    return rows / kUpRows * blocks >= kFewItems ? kUpRows : 32;
}

struct LoraLayout {
    int64_t up, down, perm, h, total;
};
LoraLayout layout(int64_t rows, int64_t adapters, int64_t k, int64_t n, int64_t rank) {
    int32_t slices, slice;
    slices_of(rows, adapters, k, &slices, &slice);
    LoraLayout o;
    o.up = 256;
    o.down = o.up + whole(most_tiles(rows, adapters, up_rows_of(rows, n)) * sizeof(Tile));
    o.perm = o.down + whole(most_tiles(rows, adapters, kDownRows) * sizeof(Tile));
    o.h = o.perm + whole(rows * 4);
    o.total = o.h + whole(slices * rows * padded_rank(rank) * 4);
    return o;
}

}  // namespace

int64_t lora_workspace(int64_t rows, int64_t adapters, int64_t k, int64_t n, int64_t rank) {
    return layout(rows, adapters, k, n, rank).total;
}

int launch_add_lora(const LoraParams &params, int dtype, int format, void *stream) {
    LoraParams p = params;
    slices_of(p.rows, p.adapters, p.k, &p.slices, &p.slice);
    p.up_rows = up_rows_of(p.rows, p.n);
    const LoraLayout o = layout(p.rows, p.adapters, p.k, p.n, p.rank);
    LoraPlan plan = {reinterpret_cast<int32_t *>(p.workspace), reinterpret_cast<Tile *>(p.workspace + o.up),
                     reinterpret_cast<Tile *>(p.workspace + o.down), reinterpret_cast<int32_t *>(p.workspace + o.perm),
                     reinterpret_cast<float *>(p.workspace + o.h)};
    // refused before anything is enqueued
    const int64_t blocks = (p.n + kUpWaves * kUpCols - 1) / (kUpWaves * kUpCols);
    const int64_t most = most_tiles(p.rows, p.adapters, p.up_rows) * blocks;
    if (most > UINT32_MAX / 2 || most_tiles(p.rows, p.adapters, kDownRows) * p.slices > UINT32_MAX / kDownThreads)
        return kTooManyWorkItems;
    const int rank = padded_rank(p.rank);
    const unsigned counters = static_cast<unsigned>(p.adapters) * 4;
    void *args[] = {&p, &plan};
    if (p.rows <= kSelfRows) {
        // A workgroup takes one pass: the first of an adapter's, or the one that a row begins where rows are fewer than adapters. Were rows
        // spread evenly, an adapter would have rows / adapters, 32 at a time if those are more than 16; workgroups for as many passes know theirs
        // at once. For more, however the rows are spread, further ones look through all of them. (An adapter's workgroup that took pass
        // after pass needed 68 us for 256 rows of one adapter among 64, 8192 -> 4096, rank 16, and 233 among 512.)
        const int64_t heads = std::min<int64_t>(p.rows, p.adapters), pass = p.rows > 16 * heads ? 32 : 16;
        const void *down = pass > 16 ? down_fn<2, true>(dtype, format, rank) : down_fn<1, true>(dtype, format, rank);
        p.parts = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(kMostParts, p.rows / (heads * 24))));
        const int64_t more = p.rows < p.adapters ? 0 : std::max<int64_t>(0, (p.rows - 1) / pass - (p.parts - 1));
        const int64_t groups = 1 + (heads * p.parts + more) * p.slices;
        if (int hip = launch_groups(down, groups, kDownThreads, args, stream, counters))
            return hip;
    } else {
        if (int hip = launch_groups(reinterpret_cast<const void *>(&lora_plan_kernel), 1, kPlanThreads, args, stream, counters))
            return hip;
        const int64_t groups = most_tiles(p.rows, p.adapters, kDownRows) * p.slices;
        const void *down = staged_fits(p, dtype, format) ? staged_fn(dtype, format, rank) : down_fn<kDownRows / 16, false>(dtype, format, rank);
        if (int hip = launch_groups(down, groups, kDownThreads, args, stream))
            return hip;
    }
    // workgroups take turns at the items: how many there are is known on the device
    const int64_t groups = std::min<int64_t>(most, kUpGroups);
    const void *up = whole_lines(p, dtype) ? up_fn<true>(dtype, rank) : up_fn<false>(dtype, rank);
    return launch_groups(up, groups, kUpThreads, args, stream);
}

}  // namespace ssu
