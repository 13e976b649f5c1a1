// Beam search's choice of continuations (ssu_beam_select), in two kernels.
//
// The score of token v behind beam i is c = score_i + (x_v - m_i) - log sum e^(x - m_i) over the allowed tokens,
// m_i the largest logit. Within a beam c has the order of the logits, so the scan needs no score: for each row (or
// share of a row) it leaves m, the sum and the first `keep` logits, in one pass over the row. The join has one workgroup
// for each request: logarithms and c in 64 bits, since scores of two beams that are near each other decide which of them
// goes on, then the first `keep` of all lists.
//
// The logits' bytes bound it. Beams at a score of -inf and ended ones are not read.
#include <algorithm>

#include "ssu_logits_device.h"

namespace ssu {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamWaves = kBeamThreads / kWaveLanes;
constexpr int kTile = kVec * kWaveLanes;  // logits per wave and access
constexpr int kInFlight = 4;              // accesses in flight per wave
constexpr float kLog2e = 1.44269504088896341f;

// Largest logit and the sum over it of a share of a row.
struct Share {
    float m, s;
};

struct BeamSplit {
    int32_t segments;  // shares per row
    int32_t tiles;     // accesses per share
    Share *shares;     // [rows, segments]
    uint64_t *keys;    // [rows, segments, keep], in order; 0: none
};

__device__ __forceinline__ float beam_score(const BeamParams &p, int64_t request, int beam) {
    return p.scores[request * p.scores_b + beam * p.scores_s];
}
__device__ __forceinline__ bool beam_ended(const BeamParams &p, int64_t request, int beam) {
    return p.finished && p.finished[request * p.finished_b + beam * p.finished_s] != 0;
}
// Whether the beam's logits count. A score of NaN or +inf spoils its request whatever they hold.
__device__ __forceinline__ bool beam_reads(float score, bool ended) {
    return !ended && score > -__builtin_inff() && score < __builtin_inff();
}

template <typename T, bool MASK>
__global__ __launch_bounds__(kBeamThreads, 4) void beam_scan_kernel(const BeamParams p, const BeamSplit sp) {
    __shared__ Share wave_shares[kBeamWaves];
    __shared__ uint64_t lists[kBeamWaves * Candidates::kList];
    __shared__ int listed;
    __shared__ float floors[kBeamWaves];  // what a wave's `keep`-th token is at least
    const int lane = threadIdx.x % kWaveLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int64_t row = blockIdx.x / sp.segments;
    const int segment = static_cast<int>(blockIdx.x % sp.segments);
    const int64_t request = row / p.beams;
    const int beam = static_cast<int>(row % p.beams);
    if (!beam_reads(beam_score(p, request, beam), beam_ended(p, request, beam)))
        return;
    if (lane == 0)
        floors[wave] = kLowest;
    if (threadIdx.x == 0)
        listed = 0;
    __syncthreads();
    const T *x_row = static_cast<const T *>(p.logits) + row * p.logits_s;
    const uint8_t *mask = MASK ? reinterpret_cast<const uint8_t *>(p.mask + row * p.mask_s) : nullptr;
    const int whole = p.vocab / kTile, tiles = (p.vocab + kTile - 1) / kTile;
    const int first = segment * sp.tiles, end = min(tiles, first + sp.tiles);
    typedef T Raw __attribute__((ext_vector_type(kVec), aligned(sizeof(T))));
    Share w = {kLowest, 0.0f};
    Candidates c = {0, 0, kLowest};
    int done = -1;  // the access whose logits have been offered before the scan

    // whole access `t`: its logits, and which of them the mask allows
    auto fetch = [&](int t, Raw *raw, uint32_t *bits) {
        const int at = t * kTile + lane * kVec;
        *bits = MASK ? mask[at / 8] : 0xFFu;
        *raw = *reinterpret_cast<const Raw *>(x_row + at);
    };
    // the row's last one, where it is not whole
    auto fetch_part = [&](int t, Raw *raw, uint32_t *bits) {
        const int at = t * kTile + lane * kVec;
        const int n = max(0, min(kVec, p.vocab - at));
        *bits = (MASK && n > 0 ? mask[at / 8] : 0xFFu) & ((1u << n) - 1);
        if (n == kVec) {
            *raw = *reinterpret_cast<const Raw *>(x_row + at);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; i++)
                (*raw)[i] = i < n ? x_row[at + i] : static_cast<T>(0.0f);
        }
    };
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
        const float top = largest(x);
        if (__ballot(top > w.m)) {
            const float m = fmaxf(w.m, wave_max(top));
            w.s *= __builtin_amdgcn_exp2f((w.m - m) * kLog2e);
            w.m = m;
        }
        float s = 0.0f;  // of this access: long chains of additions would lose digits
#pragma unroll
        for (int i = 0; i < kVec; i++)
            s += __builtin_amdgcn_exp2f((x[i] - w.m) * kLog2e);
        w.s += s;
        if (t != done && __ballot(top >= c.gate)) {
            c.offer(x, t * kTile + lane * kVec, p.keep, lane);
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
    };
    // the other waves' floors hold for this one too
    auto read_floors = [&] {
#pragma unroll
        for (int i = 0; i < kBeamWaves; i++)
            c.gate = fmaxf(c.gate, __hip_atomic_load(&floors[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP));
    };
    const int whole_end = min(end, whole);
    int t = first + wave;
    bool round = t + (kInFlight - 1) * kBeamWaves < whole_end;
    Raw raw[kInFlight];
    uint32_t bits[kInFlight];
    auto fetch_round = [&](int from) {
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            fetch(from + u * kBeamWaves, &raw[u], &bits[u]);
    };
    auto fetch_one = [&](int from) {
        if (from < whole)
            fetch(from, &raw[0], &bits[0]);
        else
            fetch_part(from, &raw[0], &bits[0]);
    };
    if (round)
        fetch_round(t);
    else if (t < end)
        fetch_one(t);
    if (t < end) {
        float best = -__builtin_inff();
#pragma unroll
        for (int u = 0; u < kInFlight; u++) {
            if (u > 0 && !round)
                break;
            float x[kVec];
            values(raw[u], bits[u], std::false_type(), x);
            best = fmaxf(best, largest(x));
        }
        c.bound(best, p.keep);
        float x[kVec];
        values(raw[0], bits[0], std::false_type(), x);
        if (c.first(x, t * kTile + lane * kVec, p.keep, lane, lists + wave * Candidates::kList)) {
            done = t;
            if (c.floor != 0 && lane == 0)
                __hip_atomic_store(&floors[wave], word_value(static_cast<uint32_t>(c.floor >> 32)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    }
    while (round) {
        read_floors();
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            take(t + u * kBeamWaves, raw[u], bits[u], std::bool_constant<!MASK>());
        t += kInFlight * kBeamWaves;
        round = t + (kInFlight - 1) * kBeamWaves < whole_end;
        if (round)
            fetch_round(t);
        else if (t < end)
            fetch_one(t);
    }
    while (t < end) {
        read_floors();
        take(t, raw[0], bits[0], std::false_type());
        t += kBeamWaves;
        if (t < end)
            fetch_one(t);
    }

    // the workgroup's sum and list
    w.s = wave_sum(w.s);
    if (lane == 0)
        wave_shares[wave] = w;
    __syncthreads();
    if (lane < p.keep && c.key != 0)
        lists[atomicAdd(&listed, 1)] = c.key;
    __syncthreads();
    const int64_t share = row * sp.segments + segment;
    if (threadIdx.x == 0) {
        Share r = {kLowest, 0.0f};
#pragma unroll
        for (int i = 0; i < kBeamWaves; i++)
            r.m = fmaxf(r.m, wave_shares[i].m);
#pragma unroll
        for (int i = 0; i < kBeamWaves; i++)
            r.s += wave_shares[i].s * __builtin_amdgcn_exp2f((wave_shares[i].m - r.m) * kLog2e);
        sp.shares[share] = r;
    }
    const int n = listed;
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
        const uint64_t key = lists[i];
        int at = 0;
        for (int j = 0; j < n; j++)
            at += lists[j] > key;
        if (at < p.keep)
            sp.keys[share * p.keep + at] = key;
    }
    for (int i = n + static_cast<int>(threadIdx.x); i < p.keep; i += kBeamThreads)
        sp.keys[share * p.keep + i] = 0;
}

// ---------------------------------------------------------------- the join

// A continuation; beams in the order of their numbers, a beam's tokens in that of their keys.
struct Continuation {
    double c;
    uint64_t key;  // its logit's (1: an ended beam's only one; 0: none)
    int32_t beam;
};
__device__ __forceinline__ bool before(const Continuation &a, const Continuation &b) {
    return a.c > b.c || (a.c == b.c && (a.beam < b.beam || (a.beam == b.beam && a.key > b.key)));
}

constexpr int kMostSegments = 64;
// Fewer rows than compute units are split, into two workgroups for each.
constexpr int kSplitBelow = 256, kSplitTo = 512;
// Lists of a request: with its rows alone below kSplitBelow it has kSplitTo + 1 for each beam at most, and a sample of them
// less than `keep` more.
constexpr int kMostSample = kSplitTo + SSU_BEAMS_MAX + SSU_TOP_MAX;
// The sample's `keep`-th stands behind the heads of at most `keep` lists, or of all if there are fewer.
constexpr int kMostChosen = SSU_TOP_MAX * SSU_TOP_MAX;

__global__ __launch_bounds__(kBeamThreads) void beam_join_kernel(const BeamParams p, const BeamSplit sp) {
    __shared__ double bias[SSU_BEAMS_MAX];  // score - log of the sum over the largest logit
    __shared__ float peak[SSU_BEAMS_MAX];   // that logit
    __shared__ uint8_t kind[SSU_BEAMS_MAX]; // 0: no candidates, 1: its logits', 2: ended
    __shared__ Continuation sample[kMostSample];
    __shared__ Continuation chosen[kMostChosen];
    __shared__ Continuation floor;
    __shared__ int bad, count;
    const int lane = threadIdx.x % kWaveLanes, wave = threadIdx.x / kWaveLanes;
    const int64_t request = blockIdx.x;
    const int64_t row0 = request * p.beams;
    const Continuation none = {-__builtin_inf(), 0, INT32_MAX};
    if (threadIdx.x == 0) {
        bad = 0;
        count = 0;
        floor = none;
    }
    __syncthreads();
    for (int i = wave; i < p.beams; i += kBeamWaves) {
        const float score = beam_score(p, request, i);
        const bool ended = beam_ended(p, request, i), reads = beam_reads(score, ended);
        if (!reads) {
            if (lane == 0) {
                if (!(score < __builtin_inff()))
                    bad = 1;
                kind[i] = ended && score > -__builtin_inff() ? 2 : 0;
                bias[i] = score;
            }
            continue;
        }
        Share s = {kLowest, 0.0f};
        if (lane < sp.segments)
            s = sp.shares[(row0 + i) * sp.segments + lane];
        float m = s.m;
#pragma unroll
        for (int d = 1; d < kWaveLanes; d *= 2)
            m = fmaxf(m, __shfl_xor(m, d));
        double sum = static_cast<double>(s.s) * __builtin_amdgcn_exp2f((s.m - m) * kLog2e);
#pragma unroll
        for (int d = 1; d < kWaveLanes; d *= 2)
            sum += __shfl_xor(sum, d);
        if (lane == 0) {
            if (sum != sum)
                bad = 1;
            kind[i] = sum > 0.0 ? 1 : 0;
            bias[i] = sum > 0.0 ? static_cast<double>(score) - log(sum) : 0.0;
            peak[i] = m;
        }
    }
    __syncthreads();
    float *out_scores = p.out_scores + request * p.keep;
    int32_t *out_parents = p.out_parents + request * p.keep, *out_tokens = p.out_tokens + request * p.keep;
    if (bad) {
        for (int i = threadIdx.x; i < p.keep; i += kBeamThreads) {
            out_scores[i] = __builtin_nanf("");
            out_parents[i] = -1;
            out_tokens[i] = -1;
        }
        return;
    }
    // place `at` of list `list` (a share of a row)
    auto continuation = [&](int list, int at) {
        const int beam = list / sp.segments, segment = list % sp.segments;
        Continuation r = none;
        if (kind[beam] == 1) {
            const uint64_t key = sp.keys[(row0 * sp.segments + list) * p.keep + at];
            if (key != 0)
                r = {bias[beam] + (static_cast<double>(key_value(key)) - peak[beam]), key, beam};
        } else if (kind[beam] == 2 && segment == 0 && at == 0) {
            r = {bias[beam], 1, beam};
        }
        return r;
    };
    // the `keep`-th of a sample, of every list's first ones: no continuation behind it is chosen
    const int lists = p.beams * sp.segments;
    const int each = min(p.keep, (p.keep + lists - 1) / lists);
    for (int i = threadIdx.x; i < lists * each; i += kBeamThreads)
        sample[i] = continuation(i / each, i % each);
    __syncthreads();
    for (int i = threadIdx.x; i < lists * each; i += kBeamThreads) {
        const Continuation mine = sample[i];
        if (mine.key == 0)
            continue;
        int at = 0;
        for (int j = 0; j < lists * each; j++)
            at += before(sample[j], mine);
        if (at == p.keep - 1)
            floor = mine;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < lists * p.keep; i += kBeamThreads) {
        const int list = i / p.keep;
        if (floor.key != 0 && before(floor, sample[list * each]))
            continue;  // its first one stands behind the floor
        const Continuation mine = continuation(list, i % p.keep);
        if (mine.key != 0 && (floor.key == 0 || !before(floor, mine)))
            chosen[atomicAdd(&count, 1)] = mine;
    }
    __syncthreads();
    const int n = count;
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
        const Continuation mine = chosen[i];
        int at = 0;
        for (int j = 0; j < n; j++)
            at += before(chosen[j], mine);
        if (at < p.keep) {
            out_scores[at] = static_cast<float>(mine.c);
            out_parents[at] = mine.beam;
            out_tokens[at] = kind[mine.beam] == 2 ? p.end_token : key_index(mine.key);
        }
    }
    for (int i = n + static_cast<int>(threadIdx.x); i < p.keep; i += kBeamThreads) {
        out_scores[i] = -__builtin_inff();
        out_parents[i] = -1;
        out_tokens[i] = -1;
    }
}

// Shares of a row and accesses per share: each has one for every wave.
void split(int64_t rows, int64_t vocab, int32_t *segments, int32_t *per) {
    const int64_t tiles = (vocab + kTile - 1) / kTile;
    int64_t s = rows < kSplitBelow ? (kSplitTo + rows - 1) / rows : 1;
    s = std::min<int64_t>({s, kMostSegments, std::max<int64_t>(1, tiles / kBeamWaves)});
    *per = static_cast<int32_t>(std::max<int64_t>(1, (tiles + s - 1) / s));
    *segments = static_cast<int32_t>(std::max<int64_t>(1, (tiles + *per - 1) / *per));
}

int64_t share_bytes(int64_t shares) { return (shares * static_cast<int64_t>(sizeof(Share)) + 255) / 256 * 256; }

template <typename T>
const void *scan_fn(bool mask) {
    return mask ? reinterpret_cast<const void *>(&beam_scan_kernel<T, true>) : reinterpret_cast<const void *>(&beam_scan_kernel<T, false>);
}

}  // namespace

int64_t beam_workspace(int64_t rows, int64_t vocab, int64_t keep) {
    int32_t s, per;
    split(rows, vocab, &s, &per);
    return share_bytes(rows * s) + rows * s * keep * 8;
}

int launch_beam_select(const BeamParams &p, int dtype, void *stream) {
    BeamSplit sp = {};
    const int64_t rows = p.batch * p.beams;
    split(rows, p.vocab, &sp.segments, &sp.tiles);
    sp.shares = reinterpret_cast<Share *>(p.workspace);
    sp.keys = reinterpret_cast<uint64_t *>(p.workspace + share_bytes(rows * sp.segments));
    const void *fn = dtype == SSU_F32   ? scan_fn<float>(p.mask != nullptr)
                     : dtype == SSU_F16 ? scan_fn<_Float16>(p.mask != nullptr)
                                        : scan_fn<__bf16>(p.mask != nullptr);
    BeamParams pc = p;
    void *args[] = {&pc, &sp};
    if (int hip = launch_groups(fn, rows * sp.segments, kBeamThreads, args, stream))
        return hip;
    return launch_groups(reinterpret_cast<const void *>(&beam_join_kernel), p.batch, kBeamThreads, args, stream);
}

}  // namespace ssu
