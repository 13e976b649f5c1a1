// Beam search's choice of continuations (ssu_beam_select), in two kernels.
//
// The score of token v behind beam i is c = score_i + (x_v - m_i) - log sum e^(x - m_i) over the allowed tokens,
// m_i the largest logit. Within a beam c has the order of the logits, so the scan needs no score: for each row (or
// share of a row) it leaves m, the sum and the first `keep` logits, in one pass over the row. The join has one workgroup
// for each request: logarithms and c in 64 bits, since scores of two beams that are near each other decide which of them
// goes on, then the first `keep` of all lists.
//
// The logits' bytes bound it, and close behind them the instructions for them (an exponential takes a quarter of the lanes
// at a time): 1601 live rows of 131072 bf16 (420 MB) take 87 us, 4.8 TB/s, 256 rows of 65536 (33 MB) 14, of which a third is the
// end of the workgroups. The join takes 5 to 6 us, of 64 beams 21. Beams at a score of -inf and ended ones are not read.
#include <algorithm>

#include "ssu_logits_device.h"

namespace ssu {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kBeamWaves = kBeamThreads / kWaveLanes;
constexpr int kTile = kVec * kWaveLanes;  // logits per wave and access
constexpr float kLog2e = 1.44269504088896341f;
constexpr int in_flight(int element) { return 16 / element; }  // accesses of a wave: 8 KiB

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

// One pass over a share of a row. Beside the wave's sum a lane keeps where its best access (eight logits) is, and the largest
// logits of that and of the second best. At least `keep` logits are not below T, the `keep`-th of the best accesses of the
// workgroup's 64 groups of four lanes; so after the pass only accesses that reach T are looked at again: a lane's best
// one, and its others only where the second best reaches T too. Of 16 kept about one lane in three workgroups does. (A list of
// each wave's first ones, kept in order during the pass, made the same 256 rows of 65536 take 28 us.)
template <typename T, bool MASK>
__global__ __launch_bounds__(kBeamThreads, 4) void beam_scan_kernel(const BeamParams p, const BeamSplit sp) {
    constexpr int kInFlight = in_flight(sizeof(T));
    constexpr int kRoom = 512;  // logits that reach T; where there are more, by equal ones, each wave finds its first ones
    __shared__ Share wave_shares[kBeamWaves];
    __shared__ uint32_t heads[kWaveLanes];
    __shared__ uint64_t list[kRoom];
    __shared__ int listed;
    const int lane = threadIdx.x % kWaveLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveLanes);
    const int64_t row = blockIdx.x / sp.segments;
    const int segment = static_cast<int>(blockIdx.x % sp.segments);
    const int64_t request = row / p.beams;
    const int beam = static_cast<int>(row % p.beams);
    const float score = beam_score(p, request, beam);
    const bool ended = beam_ended(p, request, beam);
    const T *x_row = static_cast<const T *>(p.logits) + row * p.logits_s;
    const uint8_t *mask = MASK ? reinterpret_cast<const uint8_t *>(p.mask + row * p.mask_s) : nullptr;
    const int whole = p.vocab / kTile, tiles = (p.vocab + kTile - 1) / kTile;
    const int first = segment * sp.tiles, end = min(tiles, first + sp.tiles);
    typedef T Raw __attribute__((ext_vector_type(kVec), aligned(sizeof(T))));

    // Whole access `t`: its logits, and which of them the mask allows. 16-bit logits, whose access is one instruction, go past the caches
    // (the large case above: 94 us without that); f32 ones, of two that share lines, took 19.1 us instead of 17.9 so (37 x 5 beams).
    auto fetch = [&](int t, Raw *raw, uint32_t *bits) {
        const int at = t * kTile + lane * kVec;
        *bits = MASK ? mask[at / 8] : 0xFFu;
        const Raw *x = reinterpret_cast<const Raw *>(x_row + at);
        *raw = sizeof(T) == 2 ? __builtin_nontemporal_load(x) : *x;
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
    Share w = {kLowest, 0.0f};  // m: of the wave
    float m1 = -__builtin_inff(), m2 = -__builtin_inff();  // nothing yet: below the lowest finite logit, which counts like any other
    int best_at = first + wave;
    auto take = [&](int t, const Raw &raw, uint32_t bits, auto all) {
        float x[kVec];
        values(raw, bits, all, x);
        float top = fmaxf(x[0], x[1]);
#pragma unroll
        for (int i = 2; i < kVec; i++)
            top = fmaxf(top, x[i]);
        if (__ballot(top > w.m)) {
            const float m = fmaxf(w.m, wave_max(top));
            w.s *= __builtin_amdgcn_exp2f((w.m - m) * kLog2e);
            w.m = m;
        }
        best_at = top > m1 ? t : best_at;
        m2 = __builtin_amdgcn_fmed3f(m1, m2, top);
        m1 = fmaxf(m1, top);
        float s = 0.0f;  // of this access: long chains of additions would lose digits
#pragma unroll
        for (int i = 0; i < kVec; i++)
            s += __builtin_amdgcn_exp2f((x[i] - w.m) * kLog2e);
        w.s += s;
    };
    const int whole_end = min(end, whole);
    int t = first + wave;
    Raw raw[kInFlight];
    uint32_t bits[kInFlight];
    auto fetch_round = [&] {
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            fetch(t + u * kBeamWaves, &raw[u], &bits[u]);
    };
    bool round = t + (kInFlight - 1) * kBeamWaves < whole_end;
    if (round)
        fetch_round();
    if (!beam_reads(score, ended))
        return;
    while (round) {
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            take(t + u * kBeamWaves, raw[u], bits[u], std::bool_constant<!MASK>());
        t += kInFlight * kBeamWaves;
        round = t + (kInFlight - 1) * kBeamWaves < whole_end;
        if (round)
            fetch_round();
    }
    // less than a round of whole accesses, in flight together too
    for (; t < whole_end; t += kInFlight * kBeamWaves) {
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            if (t + u * kBeamWaves < whole_end)
                fetch(t + u * kBeamWaves, &raw[u], &bits[u]);
#pragma unroll
        for (int u = 0; u < kInFlight; u++)
            if (t + u * kBeamWaves < whole_end)
                take(t + u * kBeamWaves, raw[u], bits[u], std::bool_constant<!MASK>());
    }
    if (whole < end && (whole - first) % kBeamWaves == wave) {  // the row's last, not whole
        fetch_part(whole, &raw[0], &bits[0]);
        take(whole, raw[0], bits[0], std::false_type());
    }

    // T, and the workgroup's sum
    w.s = wave_sum(w.s);
    if (lane == 0)
        wave_shares[wave] = w;
    const float four = group_max<4>(m1);
    if (lane % 4 == 0)
        heads[wave * 16 + lane / 4] = order_word(four);
    if (threadIdx.x == 0)
        listed = 0;
    __syncthreads();
    // the `keep`-th largest but for its last ten bits, which are 0, found bit by bit
    const uint32_t head = heads[lane];
    uint32_t lowest = 0;
#pragma unroll
    for (int bit = 31; bit >= 10; bit--) {
        const uint32_t t = lowest | (1u << bit);
        if (__popcll(__ballot(head >= t)) >= p.keep)
            lowest = t;
    }
    const float bound = fmaxf(word_value(lowest), kLowest);
    // the lane's logits of an access that reach T, to the list
    auto append = [&](int t, const Raw &raw, uint32_t bits) {
        float x[kVec];
        values(raw, bits, std::false_type(), x);
        uint32_t pass = 0;
#pragma unroll
        for (int i = 0; i < kVec; i++)
            pass |= x[i] >= bound && x[i] < __builtin_inff() ? 1u << i : 0;
        if (pass == 0)
            return;
        int to = atomicAdd(&listed, static_cast<int>(__popc(pass)));
#pragma unroll
        for (int i = 0; i < kVec; i++)
            if ((pass >> i) & 1) {
                if (to < kRoom)
                    list[to] = order_key(order_word(x[i]), t * kTile + lane * kVec + i);
                to++;
            }
    };
    if (m1 >= bound) {
        fetch_part(best_at, &raw[0], &bits[0]);
        append(best_at, raw[0], bits[0]);
    }
    const bool more = m2 >= bound;
    if (__ballot(more)) {
        t = first + wave;
        for (; t + (kInFlight - 1) * kBeamWaves < whole_end; t += kInFlight * kBeamWaves)
            if (more) {
                fetch_round();
#pragma unroll
                for (int u = 0; u < kInFlight; u++)
                    if (t + u * kBeamWaves != best_at)
                        append(t + u * kBeamWaves, raw[u], bits[u]);
            }
        for (; t < end; t += kBeamWaves)
            if (more && t != best_at) {
                fetch_part(t, &raw[0], &bits[0]);
                append(t, raw[0], bits[0]);
            }
    }
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
    int n = listed;
    if (n > kRoom) {
        __syncthreads();
        if (threadIdx.x == 0)
            listed = 0;
        __syncthreads();
        Candidates c = {0, static_cast<uint64_t>(order_word(bound)) << 32, bound};
        for (t = first + wave; t < end; t += kBeamWaves) {
            fetch_part(t, &raw[0], &bits[0]);
            float x[kVec];
            values(raw[0], bits[0], std::false_type(), x);
            c.offer(x, t * kTile + lane * kVec, p.keep, lane);
        }
        if (lane < p.keep && c.key != 0)
            list[atomicAdd(&listed, 1)] = c.key;
        __syncthreads();
        n = listed;
    }
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
        const uint64_t key = list[i];
        int at = 0;
        int j = 0;
        for (; j + 8 <= n; j += 8)
#pragma unroll
            for (int q = 0; q < 8; q++)
                at += list[j + q] > key;
        for (; j < n; j++)
            at += list[j] > key;
        if (at < p.keep)
            sp.keys[share * p.keep + at] = key;
    }
    if (static_cast<int>(threadIdx.x) >= n && static_cast<int>(threadIdx.x) < p.keep)
        sp.keys[share * p.keep + threadIdx.x] = 0;
}

// ---------------------------------------------------------------- the join

constexpr int kMostSegments = 64;
constexpr int kMostLists = 512;  // of a request
// Its sample: one of each list, and less than `keep` more where they are few; or about 64.
constexpr int kMostSample = kMostLists + SSU_TOP_MAX;
// The sample's `keep`-th stands behind the heads of at most `keep` lists, or of all if there are fewer.
constexpr int kMostChosen = SSU_TOP_MAX * SSU_TOP_MAX;

// A continuation's place in the order, as whole numbers: larger scores first; equal ones by beam, a beam's by their
// logits, equal logits by their places in the beam's lists, which are in the order of the tokens.
struct Place {
    uint64_t score;  // 0: none
    uint64_t rest;
};
__device__ __forceinline__ bool before(const Place &a, const Place &b) {
    return a.score > b.score || (a.score == b.score && a.rest > b.rest);
}
__device__ __forceinline__ uint64_t score_word(double c) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(c + 0.0));  // -0 and 0 are equal
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double word_score(uint64_t w) {
    return __longlong_as_double(static_cast<long long>(w >> 63 ? w & 0x7FFFFFFFFFFFFFFFull : ~w));
}
constexpr int kListBits = 11, kWordBits = 32;
static_assert(kMostSegments * SSU_TOP_MAX <= 1 << kListBits, "places in a beam's lists");
__device__ __forceinline__ uint64_t rest_word(int beam, uint32_t word, int at) {
    return (static_cast<uint64_t>(SSU_BEAMS_MAX - 1 - beam) << (kWordBits + kListBits)) | (static_cast<uint64_t>(word) << kListBits) |
           static_cast<uint64_t>((1 << kListBits) - 1 - at);
}
__device__ __forceinline__ int rest_beam(uint64_t rest) { return SSU_BEAMS_MAX - 1 - static_cast<int>(rest >> (kWordBits + kListBits)); }

// How many of places[0 .. n) stand before `mine`.
__device__ __forceinline__ int number_before(const Place *places, int n, const Place &mine) {
    int at = 0, j = 0;
    for (; j + 8 <= n; j += 8) {
        Place o[8];
#pragma unroll
        for (int q = 0; q < 8; q++)
            o[q] = places[j + q];
#pragma unroll
        for (int q = 0; q < 8; q++)
            at += before(o[q], mine);
    }
    for (; j < n; j++)
        at += before(places[j], mine);
    return at;
}

__global__ __launch_bounds__(kBeamThreads) void beam_join_kernel(const BeamParams p, const BeamSplit sp) {
    constexpr int kSamples = (kMostSample + kBeamThreads - 1) / kBeamThreads, kSampleLanes = (kMostSample + kWaveLanes - 1) / kWaveLanes;
    __shared__ double bias[SSU_BEAMS_MAX];   // score - log of the sum over the largest logit
    __shared__ float peak[SSU_BEAMS_MAX];    // that logit
    __shared__ uint8_t kind[SSU_BEAMS_MAX];  // 0: no candidates, 1: its logits', 2: ended
    __shared__ alignas(16) Place sample[kMostSample];
    __shared__ alignas(16) Place chosen[kMostChosen];
    __shared__ int32_t tokens[kMostChosen];
    __shared__ Place floor;
    __shared__ int bad, count;
    const int lane = threadIdx.x % kWaveLanes;
    const int64_t request = blockIdx.x;
    const int64_t row0 = request * p.beams;
    const int lists = p.beams * sp.segments;
    // a sample of every list's first ones, some 64 of them where the lists are few
    const int each = max((p.keep + lists - 1) / lists, min(p.keep, kWaveLanes / lists)), samples = lists * each;
    const uint64_t *keys = sp.keys + row0 * sp.segments * p.keep;
    // they are on their way while the beams' sums are joined; of beams that are not read they are anything
    uint64_t head[kSamples];
#pragma unroll
    for (int u = 0; u < kSamples; u++) {
        const int i = u * kBeamThreads + threadIdx.x;
        head[u] = i < samples ? keys[i / each * p.keep + i % each] : 0;
    }
    if (threadIdx.x == 0) {
        bad = 0;
        count = 0;
        floor = {0, 0};
    }
    __syncthreads();
    // as many lanes for each beam as a power of two holds its shares
    int width = 1;
    while (width < sp.segments)
        width *= 2;
    for (int i0 = 0; i0 < p.beams; i0 += kBeamThreads / width) {
        const int i = i0 + static_cast<int>(threadIdx.x) / width, j = lane % width;
        const bool live = i < p.beams;
        // all three are asked for at once; a share of a beam that is not read is anything
        Share s = sp.shares[(row0 + min(i, p.beams - 1)) * sp.segments + min(j, sp.segments - 1)];
        const float score = beam_score(p, request, min(i, p.beams - 1));
        const bool ended = beam_ended(p, request, min(i, p.beams - 1)), reads = beam_reads(score, ended);
        if (!reads || j >= sp.segments)
            s = {kLowest, 0.0f};
        float m = s.m;
        for (int d = 1; d < width; d *= 2)
            m = fmaxf(m, __shfl_xor(m, d));
        double sum = static_cast<double>(s.s) * __builtin_amdgcn_exp2f((s.m - m) * kLog2e);
        for (int d = 1; d < width; d *= 2)
            sum += __shfl_xor(sum, d);
        if (live && j == 0) {
            if (!(score < __builtin_inff()) || sum != sum)
                bad = 1;
            kind[i] = reads ? (sum > 0.0 ? 1 : 0) : ended && score > -__builtin_inff() ? 2 : 0;
            bias[i] = reads && sum > 0.0 ? static_cast<double>(score) - log(sum) : score;
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
    // place `at` of list `list` (a share of a row), which holds `key`
    auto continuation = [&](int list, int at, uint64_t key) {
        const int beam = list / sp.segments, segment = list - beam * sp.segments;
        if (kind[beam] == 1 && key != 0) {
            const double c = bias[beam] + (static_cast<double>(key_value(key)) - peak[beam]);
            return Place{score_word(c), rest_word(beam, static_cast<uint32_t>(key >> 32), segment * p.keep + at)};
        }
        if (kind[beam] == 2 && segment == 0 && at == 0)
            return Place{score_word(bias[beam]), rest_word(beam, 0, 0)};
        return Place{0, 0};
    };
    // A bound below the sample's `keep`-th: no score below it is chosen. Found bit by bit over the scores' leading 24 bits, by each
    // wave for itself.
    uint32_t lead[kSampleLanes];
#pragma unroll
    for (int u = 0; u < kSamples; u++) {
        const int i = u * kBeamThreads + threadIdx.x;
        if (i < samples)
            sample[i] = continuation(i / each, i % each, head[u]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSampleLanes; u++)
        lead[u] = u * kWaveLanes + lane < samples ? static_cast<uint32_t>(sample[u * kWaveLanes + lane].score >> 32) : 0;
    uint32_t bound = 0;
    auto search = [&](auto lanes) {
#pragma unroll
        for (int bit = 31; bit >= 8; bit--) {
            const uint32_t t = bound | (1u << bit);
            int above = 0;
#pragma unroll
            for (int u = 0; u < decltype(lanes)::value; u++)
                above += __popcll(__ballot(lead[u] >= t));
            bound = above >= p.keep ? t : bound;
        }
    };
    if (samples <= kWaveLanes)
        search(std::integral_constant<int, 1>());
    else if (samples <= 3 * kWaveLanes)
        search(std::integral_constant<int, 3>());
    else
        search(std::integral_constant<int, kSampleLanes>());
    // what reaches it (or, of equal scores, stands before `last`), of all lists whose first one does
    auto choose = [&](const Place &last) {
        for (int i = threadIdx.x; i < lists * p.keep; i += kBeamThreads) {
            const int list = i / p.keep;
            const Place first = sample[list * each];
            if (first.score == 0 || first.score >> 32 < bound || before(last, first))
                continue;
            const uint64_t key = keys[i];
            const Place c = continuation(list, i - list * p.keep, key);
            if (c.score != 0 && c.score >> 32 >= bound && !before(last, c)) {
                const int to = atomicAdd(&count, 1);
                if (to < kMostChosen) {
                    chosen[to] = c;
                    tokens[to] = kind[rest_beam(c.rest)] == 2 ? p.end_token : key_index(key);
                }
            }
        }
        __syncthreads();
    };
    choose(Place{0, 0});
    if (count > kMostChosen) {
        // too many scores are equal, or nearly so: the sample's `keep`-th itself is the bound
        for (int i = threadIdx.x; i < samples; i += kBeamThreads)
            if (sample[i].score != 0 && number_before(sample, samples, sample[i]) == p.keep - 1)
                floor = sample[i];
        __syncthreads();
        if (threadIdx.x == 0)
            count = 0;
        __syncthreads();
        choose(floor);
    }
    const int n = count;
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
        const Place c = chosen[i];
        const int at = number_before(chosen, n, c);
        if (at < p.keep) {
            out_scores[at] = static_cast<float>(word_score(c.score));
            out_parents[at] = rest_beam(c.rest);
            out_tokens[at] = tokens[i];
        }
    }
    for (int i = n + static_cast<int>(threadIdx.x); i < p.keep; i += kBeamThreads) {
        out_scores[i] = -__builtin_inff();
        out_parents[i] = -1;
        out_tokens[i] = -1;
    }
}

// Shares of a row and accesses per share: up to twice as many workgroups as the chip holds at once, of whole rounds of accesses; few
// rows go to shares of one access for each wave. 256 rows of 65536 bf16: 13 us in four shares, 16 in two, 21 whole; 185 of 50021 f32 with a mask
// 13.3 us in seven shares of a round, 15.4 in three; 2048 of 131072 bf16 86 in two, 97 whole, since every fourth row
// is not read and leaves its unit idle.
constexpr int64_t kGroups = 4096, kFewGroups = 512;
void split(int64_t rows, int64_t beams, int64_t vocab, int dtype, int32_t *segments, int32_t *per) {
    const int64_t tiles = (vocab + kTile - 1) / kTile, round = in_flight(dtype == SSU_F32 ? 4 : 2) * kBeamWaves;
    const int64_t most = std::min<int64_t>(kMostSegments, kMostLists / beams);
    auto whole = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    int64_t s = std::max<int64_t>(1, std::min({whole(kGroups, rows), whole(tiles, round), most}));
    int64_t each = std::max<int64_t>(1, whole(whole(tiles, s), round) * round);
    if (rows * whole(tiles, each) < kFewGroups) {
        s = std::max<int64_t>(1, std::min({whole(kFewGroups, rows), tiles / kBeamWaves, most}));
        each = std::max<int64_t>(1, whole(tiles, s));
    }
    *per = static_cast<int32_t>(each);
    *segments = static_cast<int32_t>(std::max<int64_t>(1, whole(tiles, each)));
}

int64_t share_bytes(int64_t shares) { return (shares * static_cast<int64_t>(sizeof(Share)) + 255) / 256 * 256; }

template <typename T>
const void *scan_fn(bool mask) {
    return mask ? reinterpret_cast<const void *>(&beam_scan_kernel<T, true>) : reinterpret_cast<const void *>(&beam_scan_kernel<T, false>);
}

}  // namespace

int64_t beam_workspace(int64_t rows, int64_t beams, int64_t vocab, int64_t keep, int dtype) {
    int32_t s, per;
    split(rows, beams, vocab, dtype, &s, &per);
    return share_bytes(rows * s) + rows * s * keep * 8;
}

int launch_beam_select(const BeamParams &p, int dtype, void *stream) {
    BeamSplit sp = {};
    const int64_t rows = p.batch * p.beams;
    split(rows, p.beams, p.vocab, dtype, &sp.segments, &sp.tiles);
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
