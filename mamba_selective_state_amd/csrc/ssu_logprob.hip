// Log probabilities of given tokens with entropy, rank and the top
// alternatives (ssu_token_logprobs), in one pass over the logits.
//
// With k = log2(e) / temperature and the largest logit m,
//   s = sum 2^((x - m) k),  t = sum 2^((x - m) k) (x - m) k   (over allowed tokens)
//   log p[token] = (x_token - m) / temperature - log s,  entropy = log s - t ln 2 / s.
// m is one value per wave, raised (and the sums scaled) when a logit passes it: of n accesses in no
// order about ln n do. The largest logit's own term is then 1 exactly. A reference further below costs
// digits: with one up to 2^16 times in probability below, the log probability of a token that holds nearly
// all was the difference of two numbers near 11, off by up to 2e-6 instead of 1e-7. All sums are
// f32, eight logits at a time, then a lane's, a wave's, a workgroup's.
//
// The logits' bytes bound it: 1024 x 131072 bf16 (268 MB, from HBM) take 55 us without alternatives (4.9
// TB/s). With them a wave looks at an access twice only if a logit reaches its gate: with 8 the
// same rows take 67 us, with 20 84. A row is one workgroup's (four waves that take turns at
// its accesses, four in flight each), or several workgroups' if there are few rows (see kSplitBelow).
#include <algorithm>

#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kLogprobThreads = 256;
constexpr int kLogprobWaves = kLogprobThreads / kWaveLanes;
constexpr int kVec = 8;                      // logits per lane and access
constexpr int kTile = kVec * kWaveLanes;     // per wave and access
constexpr int kInFlight = 4;                 // accesses in flight per wave
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

// One workgroup's (or, joined, one row's) sums.
struct Sums {
    float m, s, t;
    int32_t before;  // allowed tokens that stand before the given one
};

// `a` and `b` over a common reference.
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b, float k) {
    const bool first = a.m >= b.m;
    const float hi_m = first ? a.m : b.m, hi_s = first ? a.s : b.s, hi_t = first ? a.t : b.t;
    const float lo_m = first ? b.m : a.m, lo_s = first ? b.s : a.s, lo_t = first ? b.t : a.t;
    const float delta = (lo_m - hi_m) * k;  // not above 0; -inf where the references lie far apart
    const float c = __builtin_amdgcn_exp2f(delta);
    Sums r;
    r.m = hi_m;
    r.s = hi_s + c * lo_s;
    // a factor of 0 takes an infinite delta with it, but not a NaN sum
    r.t = hi_t + (c > 0.0f ? c * (lo_t + delta * lo_s) : 0.0f * lo_t);
    r.before = a.before + b.before;
    return r;
}

template <typename T>
struct RowView {
    const T *x;
    const uint8_t *mask;  // bit i of byte j allows token 8 j + i; or null
    float k;              // log2(e) / temperature
    float inv;            // 1 / temperature
    bool bad;             // the temperature is not above 0
    int64_t token;
    bool inside;  // the token lies in the vocabulary
};

template <typename T>
__device__ __forceinline__ RowView<T> row_view(const LogprobParams &p, int64_t row) {
    RowView<T> v;
    v.x = static_cast<const T *>(p.logits) + row * p.logits_s;
    v.mask = p.mask ? reinterpret_cast<const uint8_t *>(p.mask + row * p.mask_s) : nullptr;
    const float temp = p.temperature ? p.temperature[row * p.temp_s] : 1.0f;
    v.bad = !(temp > 0.0f);
    // finite and above 0, so that 0 and -inf times it stay what they are
    v.k = fminf(fmaxf(1.44269504088896341f / temp, 1.1754944e-38f), -kLowest);
    v.inv = fminf(1.0f / temp, -kLowest);
    v.token = p.tokens_i64 ? static_cast<const int64_t *>(p.tokens)[row * p.tokens_s]
                           : static_cast<const int32_t *>(p.tokens)[row * p.tokens_s];
    v.inside = v.token >= 0 && v.token < p.vocab;
    return v;
}

// The given token's logit (-inf if it is not allowed) and how many allowed logits equal it at
// lower indices of its access: the scan takes of that access only the logits above it. Eight lanes
// fetch the access's logits together.
template <typename T>
__device__ __forceinline__ void token_logit(const RowView<T> &v, int vocab, int lane, float *mine, int *equal) {
    const int token = v.inside ? static_cast<int>(v.token) : 0;
    const int at = token / kVec * kVec + lane;
    const bool mine_lane = lane < kVec && at < vocab && v.inside;
    float x = -__builtin_inff();
    if (mine_lane) {
        x = widen(v.x[at]);
        if (v.mask && !((v.mask[at / 8] >> (at % 8)) & 1))
            x = -__builtin_inff();
    }
    *mine = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), token % kVec));
    *equal = __popcll(__ballot(mine_lane && at < token && x == *mine));
}

// Writes a row's results (one thread; `mine`: the token's logit, `equal`: see token_logit, `logs`:
// log s).
__device__ __forceinline__ void write_row(const LogprobParams &p, int64_t row, const Sums &r, float mine, int equal, float inv,
                                          bool bad, float logs) {
    const bool have = mine > -__builtin_inff();
    const float nan = __builtin_nanf("");
    p.logprob[row] = bad ? nan : have ? (mine - r.m) * inv - logs : -__builtin_inff();
    p.entropy[row] = bad ? nan : r.s > 0.0f ? fmaxf(logs - r.t / r.s * 0.693147180559945309f, 0.0f) : 0.0f;
    p.rank[row] = bad || !have ? -1 : r.before + equal;
}

__device__ __forceinline__ void write_alternative(const LogprobParams &p, int64_t row, int place, uint64_t key, const Sums &r,
                                                  float inv, bool bad, float logs) {
    const bool have = !bad && key != 0;
    p.top_tokens[row * p.top + place] = have ? key_index(key) : -1;
    p.top_logprobs[row * p.top + place] = bad    ? __builtin_nanf("")
                                          : have ? (key_value(key) - r.m) * inv - logs
                                                 : -__builtin_inff();
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

struct Split {
    int32_t segments;  // workgroups per row
    int32_t tiles;     // tiles per segment
    uint32_t *tickets; // [rows]: workgroups of the row that are done; 0 between calls
    Sums *sums;        // [rows, segments]
    uint64_t *keys;    // [rows, segments, top]
};

constexpr int kMostSegments = 64;
// Fewer rows than compute units are split, into two workgroups for each. f32, vocabulary 131072, no
// alternatives and 20, in us: 1 row split 6.3 and 12.3, whole 16.5 and 42.7; 64 rows 10.0 and 23.8,
// 17.5 and 45.5; 200 rows 22.0 and 42.9, 21.1 and 47.5; 400 rows 38.9 and 60.9, 32.8 and 57.5. One
// workgroup for each instead of two: 64 rows 10.3 and 27.3, four 12.5 and 23.1.
constexpr int kSplitBelow = 256, kSplitTo = 512;
constexpr int kTicketBytes = SSU_LOGPROB_ZEROED_BYTES;  // of the workspace, at its start
static_assert(4 * kSplitBelow <= kTicketBytes, "a ticket for each row that is split");
constexpr int kMergeCand = kMostSegments * SSU_TOP_MAX;  // keys of a row's segments, at most

template <typename T, bool MASK, bool TOP>
__global__ __launch_bounds__(kLogprobThreads, 4) void logprob_kernel(const LogprobParams p, const Split sp) {
    __shared__ Sums wave_sums[kLogprobWaves];
    __shared__ Sums total;
    __shared__ uint64_t merged[TOP ? kMergeCand : 1];
    __shared__ uint64_t floor;  // of the joined segments
    __shared__ int merged_n, last;
    __shared__ float floors[kLogprobWaves];  // what a wave's top-th token is at least
    const int lane = threadIdx.x % kWaveLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int64_t row = blockIdx.x / sp.segments;
    const int segment = static_cast<int>(blockIdx.x % sp.segments);
    if constexpr (TOP) {
        if (lane == 0)
            floors[wave] = kLowest;
        __syncthreads();
    }
    const RowView<T> v = row_view<T>(p, row);
    const int whole = p.vocab / kTile, tiles = (p.vocab + kTile - 1) / kTile;
    const int first = segment * sp.tiles, end = min(tiles, first + sp.tiles);
    typedef T Raw __attribute__((ext_vector_type(kVec), aligned(sizeof(T))));
    Sums w = {kLowest, 0.0f, 0.0f, 0};
    Candidates c = {0, 0, kLowest};
    int done = -1;  // the access whose logits have been offered before the scan

    // whole tile `t`: its logits, and which of them the mask allows
    auto fetch = [&](int t, Raw *raw, uint32_t *bits) {
        const int at = t * kTile + lane * kVec;
        *bits = MASK ? v.mask[at / 8] : 0xFFu;
        *raw = *reinterpret_cast<const Raw *>(v.x + at);
    };
    // the row's last tile, where it is not whole
    auto fetch_part = [&](int t, Raw *raw, uint32_t *bits) {
        const int at = t * kTile + lane * kVec;
        const int n = max(0, min(kVec, p.vocab - at));
        *bits = (MASK && n > 0 ? v.mask[at / 8] : 0xFFu) & ((1u << n) - 1);
        if (n == kVec) {
            *raw = *reinterpret_cast<const Raw *>(v.x + at);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; i++)
                (*raw)[i] = i < n ? v.x[at + i] : static_cast<T>(0.0f);
        }
    };
    // what this wave reads first is on its way before the token's own logit is asked for
    using Every = std::bool_constant<!MASK>;
    const int whole_end = min(end, whole);
    int t = first + wave;
    bool round = t + (kInFlight - 1) * kLogprobWaves < whole_end;
    Raw raw[kInFlight];
    uint32_t bits[kInFlight];
    auto fetch_round = [&](int from, Raw *r, uint32_t *b) {
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            fetch(from + u * kLogprobWaves, &r[u], &b[u]);
    };
    auto fetch_one = [&](int from, Raw *r, uint32_t *b) {
        if (from < whole)
            fetch(from, r, b);
        else
            fetch_part(from, r, b);
    };
    if (round)
        fetch_round(t, raw, bits);
    else if (t < end)
        fetch_one(t, raw, bits);
    float mine;
    int equal;
    token_logit(v, p.vocab, lane, &mine, &equal);
    const bool counted = mine > -__builtin_inff();
    const int token = counted ? static_cast<int>(v.token) : 0;
    // logits above it stand before the token: at lower indices the equal ones too
    const float mine_low = counted ? next_below(mine) : __builtin_inff(), mine_high = counted ? mine : __builtin_inff();

    auto values = [&](const Raw &raw, uint32_t bits, auto all, float x[kVec]) {
#pragma unroll
        for (int i = 0; i < kVec; i++) {
            x[i] = widen(raw[i]);
            if constexpr (!decltype(all)::value)
                x[i] = (bits >> i) & 1 ? x[i] : -__builtin_inff();
        }
    };
    auto largest = [&](const float x[kVec]) {
        float a = fmaxf(x[0], x[1]);
#pragma unroll
        for (int i = 2; i < kVec; i++)
            a = fmaxf(a, x[i]);
        return a;
    };
    auto take = [&](int t, const Raw &raw, uint32_t bits, auto all) {
        float x[kVec];
        values(raw, bits, all, x);
        const int at = t * kTile + lane * kVec;
        const float top = largest(x);
        if (__ballot(top > w.m)) {
            const float m = fmaxf(w.m, wave_max(top));
            const float delta = (w.m - m) * v.k, f = __builtin_amdgcn_exp2f(delta);
            w.t = f > 0.0f ? f * (w.t + delta * w.s) : 0.0f * w.t;
            w.s *= f;
            w.m = m;
        }
        float low = mine_high;
        if (at + kVec <= token)
            low = mine_low;
        int before = 0;
        float s = 0.0f, q = 0.0f;  // of this access: long chains of additions would lose digits
#pragma unroll
        for (int i = 0; i < kVec; i++) {
            const float d = (x[i] - w.m) * v.k;
            const float e = __builtin_amdgcn_exp2f(d);
            s += e;
            q = fmaf(e, fmaxf(d, -1e30f), q);  // d may be -inf
            before += __popcll(__ballot(x[i] > low));
        }
        w.s += s;
        w.t += q;
        w.before += before;
        if constexpr (TOP) {
            if (t != done && __ballot(top >= c.gate)) {
                c.offer(x, at, p.top, lane);
                const uint32_t word = static_cast<uint32_t>(c.floor >> 32);
                if (word != 0) {
                    const float value = word_value(word);
                    if (lane == 0)
                        __hip_atomic_store(&floors[wave], value, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                    // accesses come in the order of their indices: what only equals a token of
                    // this wave stays behind it from here on (a bound's key has no index)
                    if (static_cast<uint32_t>(c.floor) != 0)
                        c.gate = fmaxf(c.gate, next_above(value));
                }
            }
        }
    };
    // the other waves' floors hold for this one too
    auto read_floors = [&] {
        if constexpr (TOP) {
#pragma unroll
            for (int i = 0; i < kLogprobWaves; i++)
                c.gate = fmaxf(c.gate, __hip_atomic_load(&floors[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP));
        }
    };
    if (TOP && t < end) {
        float best = -__builtin_inff();
#pragma unroll
        for (int u = 0; u < kInFlight; u++) {
            if (u > 0 && !round)
                break;
            float x[kVec];
            values(raw[u], bits[u], std::false_type(), x);
            best = fmaxf(best, largest(x));
        }
        c.bound(best, p.top);
        float x[kVec];
        values(raw[0], bits[0], std::false_type(), x);
        if (c.first(x, t * kTile + lane * kVec, p.top, lane, merged + wave * Candidates::kList)) {
            done = t;
            if (c.floor != 0 && lane == 0)
                __hip_atomic_store(&floors[wave], word_value(static_cast<uint32_t>(c.floor >> 32)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    }
    while (round) {
        read_floors();
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            take(t + u * kLogprobWaves, raw[u], bits[u], Every());
        t += kInFlight * kLogprobWaves;
        round = t + (kInFlight - 1) * kLogprobWaves < whole_end;
        if (round)
            fetch_round(t, raw, bits);
        else if (t < end)
            fetch_one(t, raw, bits);
    }
    while (t < end) {
        read_floors();
        take(t, raw[0], bits[0], std::false_type());
        t += kLogprobWaves;
        if (t < end)
            fetch_one(t, raw, bits);
    }

    // the workgroup's sums and candidates
    w.s = wave_sum(w.s);
    w.t = wave_sum(w.t);
    if (lane == 0) {
        wave_sums[wave] = w;
    }
    if (threadIdx.x == 0)
        merged_n = 0;
    __syncthreads();
    Sums r = wave_sums[0];
#pragma unroll
    for (int i = 1; i < kLogprobWaves; i++)
        r = join(r, wave_sums[i], v.k);
    // the first p.top of merged[0 .. n) to their places
    auto place = [&](int n, auto out) {
        for (int i = threadIdx.x; i < n; i += kLogprobThreads) {
            const uint64_t key = merged[i];
            int at = 0;
            int j = 0;
            for (; j + 8 <= n; j += 8)
#pragma unroll
                for (int q = 0; q < 8; q++)
                    at += merged[j + q] > key;
            for (; j < n; j++)
                at += merged[j] > key;
            if (at < p.top)
                out(at, key);
        }
        for (int i = n + static_cast<int>(threadIdx.x); i < p.top; i += kLogprobThreads)
            out(i, static_cast<uint64_t>(0));
    };
    if constexpr (TOP) {
        if (lane < p.top && c.key != 0)
            merged[atomicAdd(&merged_n, 1)] = c.key;
        __syncthreads();
    }
    const bool bad_sum = r.s != r.s;
    if (sp.segments == 1) {
        const bool bad = v.bad || bad_sum;
        const float logs = __builtin_amdgcn_logf(r.s) * 0.693147180559945309f;
        if (threadIdx.x == 0)
            write_row(p, row, r, mine, equal, v.inv, bad, logs);
        if constexpr (TOP)
            place(merged_n, [&](int at, uint64_t key) { write_alternative(p, row, at, key, r, v.inv, bad, logs); });
        return;
    }

    // Several workgroups per row: each leaves its share in the workspace, and the last one
    // to do so joins them. Shares are written and read with device-scope accesses, which go
    // past the dies' own caches, and complete before the ticket is drawn; a release fence, which
    // writes a whole L2 back, took 40 us over 518 workgroups.
    const int64_t base = row * sp.segments;
    auto put = [](auto *at, auto value) { __hip_atomic_store(at, value, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    auto get = [](auto *at) { return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    if (threadIdx.x == 0) {
        Sums *at = sp.sums + base + segment;
        put(&at->m, r.m);
        put(&at->s, r.s);
        put(&at->t, r.t);
        put(&at->before, r.before);
    }
    if constexpr (TOP)
        place(merged_n, [&](int at, uint64_t key) { put(sp.keys + (base + segment) * p.top + at, key); });
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's stores are complete
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t done = __hip_atomic_fetch_add(sp.tickets + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = done + 1 == static_cast<uint32_t>(sp.segments);
        if (last)
            put(sp.tickets + row, 0u);
        merged_n = 0;
    }
    __syncthreads();
    if (!last)
        return;
    if (wave == 0) {
        Sums mine_part = {kLowest, 0.0f, 0.0f, 0};
        if (lane < sp.segments) {
            Sums *at = sp.sums + base + lane;
            mine_part = {get(&at->m), get(&at->s), get(&at->t), get(&at->before)};
        }
        // the order of the joins is fixed: by lane
#pragma unroll
        for (int d = 1; d < kWaveLanes; d *= 2) {
            const Sums o = {__shfl_xor(mine_part.m, d), __shfl_xor(mine_part.s, d), __shfl_xor(mine_part.t, d),
                            __shfl_xor(mine_part.before, d)};
            mine_part = lane & d ? join(o, mine_part, v.k) : join(mine_part, o, v.k);
        }
        if (lane == 0)
            total = mine_part;
    }
    if constexpr (TOP) {
        // every thread's keys, on their way while the floor is found
        constexpr int kMost = kMostSegments * SSU_TOP_MAX / kLogprobThreads;
        uint64_t keys[kMost];
#pragma unroll
        for (int i = 0; i < kMost; i++) {
            const int at = i * kLogprobThreads + threadIdx.x;
            keys[i] = at < sp.segments * p.top ? get(sp.keys + base * p.top + at) : 0;
        }
        // the top-th of 64 of them, each segment's first ones, is behind no alternative
        if (wave == 1) {
            const int each = min(p.top, kWaveLanes / sp.segments);
            const uint64_t k = lane < each * sp.segments ? get(sp.keys + (base + lane / each) * p.top + lane % each) : 0;
            int at = 0;
            for (int j = 0; j < kWaveLanes; j++) {
                const uint64_t o = (static_cast<uint64_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(k >> 32), j)) << 32) |
                                   static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<uint32_t>(k), j));
                at += o > k || (o == k && j < lane);
            }
            if (at == p.top - 1)
                floor = k;  // 0 where there are fewer
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMost; i++)
            if (keys[i] != 0 && keys[i] >= floor)
                merged[atomicAdd(&merged_n, 1)] = keys[i];
    }
    __syncthreads();
    r = total;
    const bool bad = v.bad || r.s != r.s;
    const float logs = __builtin_amdgcn_logf(r.s) * 0.693147180559945309f;
    if (threadIdx.x == 0)
        write_row(p, row, r, mine, equal, v.inv, bad, logs);
    if constexpr (TOP)
        place(merged_n, [&](int at, uint64_t key) { write_alternative(p, row, at, key, r, v.inv, bad, logs); });
}

template <typename T>
const void *logprob_fn(bool mask, bool top) {
    return mask ? (top ? reinterpret_cast<const void *>(&logprob_kernel<T, true, true>)
                       : reinterpret_cast<const void *>(&logprob_kernel<T, true, false>))
                : (top ? reinterpret_cast<const void *>(&logprob_kernel<T, false, true>)
                       : reinterpret_cast<const void *>(&logprob_kernel<T, false, false>));
}

// Segments of a row and tiles per segment.
void split(int64_t rows, int64_t vocab, int32_t *segments, int32_t *per) {
    const int64_t tiles = (vocab + kTile - 1) / kTile;
    int64_t s = rows < kSplitBelow ? (kSplitTo + rows - 1) / rows : 1;
    // a segment has a tile for each wave
    s = std::min<int64_t>({s, kMostSegments, std::max<int64_t>(1, tiles / kLogprobWaves)});
    *per = static_cast<int32_t>(std::max<int64_t>(1, (tiles + s - 1) / s));
    *segments = static_cast<int32_t>(std::max<int64_t>(1, (tiles + *per - 1) / *per));
}

}  // namespace

// The tickets come first, at a fixed size: what one call uses for shares is never
// another's ticket.
int64_t logprobs_workspace(int64_t rows, int64_t vocab, int64_t top) {
    int32_t s, per;
    split(rows, vocab, &s, &per);
    return s == 1 ? 0 : kTicketBytes + rows * s * static_cast<int64_t>(sizeof(Sums) + 8 * top);
}

int launch_logprobs(const LogprobParams &p, int dtype, void *stream) {
    Split sp = {};
    split(p.rows, p.vocab, &sp.segments, &sp.tiles);
    if (sp.segments > 1) {
        sp.tickets = reinterpret_cast<uint32_t *>(p.workspace);
        sp.sums = reinterpret_cast<Sums *>(p.workspace + kTicketBytes);
        sp.keys = reinterpret_cast<uint64_t *>(sp.sums + p.rows * sp.segments);
    }
    const bool mask = p.mask != nullptr, top = p.top > 0;
    const void *fn = dtype == SSU_F32   ? logprob_fn<float>(mask, top)
                     : dtype == SSU_F16 ? logprob_fn<_Float16>(mask, top)
                                        : logprob_fn<__bf16>(mask, top);
    LogprobParams pc = p;
    void *args[] = {&pc, &sp};
    return launch_groups(fn, p.rows * sp.segments, kLogprobThreads, args, stream);
}

}  // namespace ssu
