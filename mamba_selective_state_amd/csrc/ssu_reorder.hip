// Sequence states after a beam search's choice (ssu_reorder_states).
//
// The first successor of a beam goes on in its slot; only further ones are copied, into the slots of beams without a
// successor. As many are left as are needed, and nothing reads them, so the copies have no order: every workgroup
// finds them for itself from the request's row of parents (a ballot for each beam) and copies its piece of the slot for each. The
// bytes of the copied slots bound it, read and written once: 24 slots of 2.1 MB in each of eight layers (829 MB) take 144 us, 5.7 TB/s,
// some of it from the last-level cache; a copy of 1 GiB reaches 5.2. A piece is what the workgroup's lanes have in flight together, 16 KiB.
#include <algorithm>

#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kReorderThreads = 256;
constexpr int kReorderWaves = kReorderThreads / kWaveLanes;
constexpr int kReorderInFlight = 4;  // accesses of 16 bytes in flight per lane
constexpr int64_t kReorderRound = kReorderThreads * 16 * kReorderInFlight;  // bytes a workgroup moves at a time

typedef u32x4 Any4 __attribute__((aligned(1)));

// An index as a slot or beam number; -1 where it is none of [0, end).
__device__ __forceinline__ int number_of(const void *base, bool i64, int64_t at, int64_t end) {
    const int64_t v = i64 ? static_cast<const int64_t *>(base)[at] : static_cast<const int32_t *>(base)[at];
    return v >= 0 && v < end ? static_cast<int>(v) : -1;
}

__global__ __launch_bounds__(kReorderThreads) void reorder_kernel(const ReorderParams p) {
    __shared__ int free_slots[kReorderWaves][kWaveLanes];
    const int lane = threadIdx.x % kWaveLanes, wave = threadIdx.x / kWaveLanes;
    const int pieces = p.first_piece[p.count];
    const int64_t request = blockIdx.x / pieces;
    const int piece = static_cast<int>(blockIdx.x % pieces);
    const bool mine = lane < p.beams;
    int parent = -1, slot = -1;
    if (mine) {
        parent = number_of(p.parents, p.parents_i64, request * p.parents_b + lane * p.parents_s, p.beams);
        slot = number_of(p.slots, p.slots_i64, request * p.slots_b + lane * p.slots_s, INT32_MAX);
    }
    // beams that go on, and whether this lane's successor is the first of its parent
    uint64_t used = 0;
    bool stays = false;
    for (int i = 0; i < p.beams; i++) {
        const uint64_t of = __ballot(parent == i);
        if (of == 0)
            continue;
        used |= 1ull << i;
        stays = stays || __builtin_ctzll(of) == lane;
    }
    const uint64_t below = (1ull << lane) - 1;
    const uint64_t free = __ballot(mine) & ~used, moves = __ballot(mine && !stays);
    if ((free >> lane) & 1)
        free_slots[wave][__popcll(free & below)] = slot;
    wave_lds_fence();
    const int from = __shfl(slot, max(parent, 0));
    const int to = stays || !mine ? from : free_slots[wave][__popcll(moves & below)];
    if (piece == 0 && wave == 0 && mine) {
        const int64_t at = request * p.out_b + lane;
        if (p.out_i64)
            static_cast<int64_t *>(p.out)[at] = to;
        else
            static_cast<int32_t *>(p.out)[at] = to;
    }
    int pool = 0;
    while (pool + 1 < p.count && piece >= p.first_piece[pool + 1])
        pool++;
    if (p.count == 0)
        return;
    const ReorderPool q = p.pool[pool];
    const int64_t begin = static_cast<int64_t>(piece - p.first_piece[pool]) * p.piece, end = min(q.bytes, begin + p.piece);
    uint64_t todo = __ballot(mine && !stays && parent >= 0);
    while (todo) {
        const int j = __builtin_ctzll(todo);
        todo &= todo - 1;
        const int s = __builtin_amdgcn_readlane(from, j), d = __builtin_amdgcn_readlane(to, j);
        if (s < 0 || d < 0 || s >= q.slots || d >= q.slots)
            continue;
        const uint8_t *src = q.base + s * q.stride;
        uint8_t *dst = q.base + d * q.stride;
        int64_t at = begin + threadIdx.x * 16;
        for (; at + (kReorderInFlight - 1) * kReorderThreads * 16 + 16 <= end; at += kReorderRound) {
            u32x4 v[kReorderInFlight];
#pragma unroll
            for (int u = 0; u < kReorderInFlight; u++)
                v[u] = *reinterpret_cast<const Any4 *>(src + at + u * kReorderThreads * 16);
#pragma unroll
            for (int u = 0; u < kReorderInFlight; u++)
                *reinterpret_cast<Any4 *>(dst + at + u * kReorderThreads * 16) = v[u];
        }
        for (; at < end; at += kReorderThreads * 16) {
            if (at + 16 <= end) {
                *reinterpret_cast<Any4 *>(dst + at) = *reinterpret_cast<const Any4 *>(src + at);
            } else {
                for (int64_t i = at; i < end; i++)
                    dst[i] = src[i];
            }
        }
    }
}

}  // namespace

int plan_reorder(ReorderParams &p) {
    p.piece = kReorderRound;
    int64_t pieces = 0;
    for (int i = 0; i < p.count; i++) {
        p.first_piece[i] = static_cast<int32_t>(pieces);
        pieces += (p.pool[i].bytes + p.piece - 1) / p.piece;
        if (pieces > INT32_MAX)
            return kTooManyWorkItems;
    }
    pieces = std::max<int64_t>(pieces, 1);  // the slots are written all the same
    p.first_piece[p.count] = static_cast<int32_t>(pieces);
    return groups_fit(p.batch * pieces, kReorderThreads) ? 0 : kTooManyWorkItems;
}

int launch_reorder(const ReorderParams &params, void *stream) {
    ReorderParams p = params;
    void *args[] = {&p};
    return launch_groups(reinterpret_cast<const void *>(&reorder_kernel), p.batch * p.first_piece[p.count], kReorderThreads, args, stream);
}

}  // namespace ssu
