// Rows to MXFP8 / MXFP4 (ssu_mx_quantize) and the product of such rows with
// MXFP4 weights (ssu_mx_linear) on the block-scaled matrix instructions.
//
// Operand layouts of those instructions (checked on the device): lane l of a
// wave holds row r = l % R of its operand (R = 16 or 32) and k group g = l / R;
// E2M1 codes: k = 32 g .. 32 g + 31 in four registers; E4M3 codes: k = 16 g ..
// 16 g + 15 in the first four and as many, K / 2 further on, in the last four
// (K: the instruction's depth); the scale byte, one of a register's four, is that
// of k block g. The first operand's rows are the result's rows (register i of lane
// l: row i % 4 + 8 (i / 4) + 4 (l / 32) with R = 32, i + 4 (l / 16) with R = 16), the
// second operand's rows its columns (l % R). The weights go first: a lane then holds
// four neighbouring outputs of one activation row.
//
// Which k block the instruction calls g is free as long as both operands and
// both scales agree. The tiled kernel gives group h of step s the block STEPS h + s
// of its K tile, so that one register holds a lane's scale bytes of all steps
// and each step names its byte.
#include <algorithm>

#include "ssu_layer_device.h"

namespace ssu {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kE4M3 = 0, kE2M1 = 4;  // the instructions' format numbers

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x8 wide(i32x4 lo, i32x4 hi) {
    return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
}
__device__ __forceinline__ i32x8 wide(i32x4 lo) { return i32x8{lo.x, lo.y, lo.z, lo.w, 0, 0, 0, 0}; }
__device__ __forceinline__ i32x8 wide(i32x8 v) { return v; }

// Four lanes per block of 32 values, eight each.
template <typename T, int FORMAT>
__global__ __launch_bounds__(kQuantThreads) void mx_quantize_rows_kernel(const T *src, int64_t stride, int64_t rows,
                                                                         int32_t k, uint8_t *codes, uint8_t *scales) {
    const int64_t eighths = k / 8;  // per row
    const int64_t total = rows * eighths;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQuantThreads;
    // four lanes of a block are live or not together: a row is a multiple of four eighths
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x; i < total; i += step) {
        const int64_t row = i / eighths, at = (i % eighths) * 8;
        float v[8];
        load8(src + row * stride + at, v);
        uint32_t code[2];
        const uint32_t s = mx_block<FORMAT>(v, code);
        store_codes<FORMAT>(codes + row * (FORMAT == SSU_FORMAT_MXFP4 ? k / 2 : k), at, code);
        if (i % 4 == 0)
            scales[i / 4] = static_cast<uint8_t>(s);
    }
}

// Adds the bias of outputs n .. n + 3.
template <typename OT>
__device__ __forceinline__ f32x4 add_bias(const MxParams &p, int n, f32x4 v) {
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int at = min(n + i, p.n - 1);
            v[i] += p.bias_f32 ? static_cast<const float *>(p.bias)[at] : widen(static_cast<const OT *>(p.bias)[at]);
        }
    }
    return v;
}

// Four neighbouring outputs of row m, from n on.
template <typename OT>
__device__ __forceinline__ void store_out4(const MxParams &p, int m, int n, f32x4 v) {
    if (m >= p.m || n >= p.n)
        return;
    OT *dst = static_cast<OT *>(p.out) + m * p.out_s + n;
    typedef OT Vec __attribute__((ext_vector_type(4), aligned(sizeof(OT))));
    Vec r;
#pragma unroll
    for (int i = 0; i < 4; i++)
        r[i] = narrow<OT>(v[i]);
    if (n + 4 <= p.n) {
        *reinterpret_cast<Vec *>(dst) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 3; i++)
            if (n + i < p.n)
                dst[i] = r[i];
    }
}

// ---------------------------------------------------------------- few rows
//
// The weights' bytes bound it. A workgroup takes 16 outputs of up to 16 rows; its waves split
// k and join their sums in LDS.

constexpr int kStreamWaves = 8;
constexpr int kStreamRows = 16;  // weight rows per workgroup
constexpr int kStreamSteps = 4;  // 128-deep steps of a round, whose loads are in flight together (see round_scales)

// The scale bytes of a lane's blocks first + 4 s + g (s = 0..3) of a row, each in the lowest byte of
// its word; 0 past the last block. One 16-byte access for the four lanes of a row: a byte
// for each lane and step took a third of the kernel's time.
__device__ __forceinline__ i32x4 round_scales(const uint8_t *row, int first, int blocks, int g) {
    typedef int Vec __attribute__((ext_vector_type(4), aligned(1)));
    i32x4 v = {};
    if (first + 16 <= blocks) {
        v = *reinterpret_cast<const Vec *>(row + first);
    } else {
#pragma unroll
        for (int s = 0; s < 4; s++)
            if (first + 4 * s + g < blocks)
                v[s] = row[first + 4 * s + g] << (8 * g);
    }
#pragma unroll
    for (int s = 0; s < 4; s++)
        v[s] = static_cast<int>(static_cast<uint32_t>(v[s]) >> (8 * g));
    return v;
}

// FT: the activations' float type when this kernel quantises them (at most kMxFuseRows rows),
// else void.
template <typename OT, int FORMAT, typename FT>
__global__ __launch_bounds__(kStreamWaves * 64) void mx_stream_kernel(const MxParams p) {
    constexpr bool kFuse = !std::is_void_v<FT>;
    constexpr int kChunk = kStreamSteps * 128;  // k values per round
    constexpr int kRowBytes = FORMAT == SSU_FORMAT_MXFP8 ? kChunk : kChunk / 2;
    __shared__ f32x4 sums[kStreamWaves][64];
    __shared__ alignas(16) uint8_t qcodes[kFuse ? kStreamWaves : 1][kMxFuseRows][kRowBytes];
    __shared__ uint8_t qscales[kFuse ? kStreamWaves : 1][kMxFuseRows][kChunk / 32];
    const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int r = l % 16, g = l / 16;
    const int n0 = static_cast<int>(blockIdx.x) * kStreamRows;
    // rows past the end read the last row; their results are not stored
    const int64_t wrow = min(n0 + r, p.n - 1);
    const uint8_t *w = p.w + wrow * p.w_s, *ws = p.w_scale + wrow * p.ws_s;
    const int blocks = p.k / 32;
    const int steps = (blocks + 3) / 4;
    const int rounds = (steps + kStreamSteps - 1) / kStreamSteps;
    f32x4 acc = {};
    for (int round = wave; round < rounds; round += kStreamWaves) {
        const int first = round * kStreamSteps;
        i32x4 wv[kStreamSteps];
#pragma unroll
        for (int s = 0; s < kStreamSteps; s++) {
            const int b = (first + s) * 4 + g;
            wv[s] = b < blocks ? *reinterpret_cast<const i32x4 *>(w + static_cast<int64_t>(b) * 16) : i32x4{};
        }
        const i32x4 wsv = round_scales(ws, first * 4, blocks, g);
        if constexpr (kFuse) {
            // this wave's own slice of every activation row, quantised for itself
            const int at = round * kChunk + l * 8;
            for (int m = 0; m < p.m; m++) {
                float v[8] = {};
                if (at < p.k)
                    load8(static_cast<const FT *>(p.x) + m * p.x_s + at, v);
                uint32_t code[2];
                const uint32_t sc = mx_block<FORMAT>(v, code);
                store_codes<FORMAT>(qcodes[wave][m], l * 8, code);
                if (l % 4 == 0)
                    qscales[wave][m][l / 4] = static_cast<uint8_t>(sc);
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        const int m = min(r, p.m - 1);
        const uint8_t *a = kFuse ? nullptr : p.a + m * p.a_s;
        i32x4 asv = {};
        if constexpr (!kFuse)
            asv = round_scales(p.a_scale + m * p.as_s, first * 4, blocks, g);
#pragma unroll
        for (int s = 0; s < kStreamSteps; s++) {
            i32x8 av;
            int as;
            if constexpr (kFuse) {
                if constexpr (FORMAT == SSU_FORMAT_MXFP8)
                    av = wide(*reinterpret_cast<const i32x4 *>(&qcodes[wave][m][s * 128 + 16 * g]),
                              *reinterpret_cast<const i32x4 *>(&qcodes[wave][m][s * 128 + 64 + 16 * g]));
                else
                    av = wide(*reinterpret_cast<const i32x4 *>(&qcodes[wave][m][s * 64 + 16 * g]));
                as = qscales[wave][m][s * 4 + g];
            } else {
                const int b = (first + s) * 4;
                as = asv[s];
                if constexpr (FORMAT == SSU_FORMAT_MXFP8) {
                    const i32x4 lo = b + g / 2 < blocks ? *reinterpret_cast<const i32x4 *>(a + static_cast<int64_t>(b) * 32 + 16 * g) : i32x4{};
                    const i32x4 hi = b + 2 + g / 2 < blocks ? *reinterpret_cast<const i32x4 *>(a + static_cast<int64_t>(b) * 32 + 64 + 16 * g) : i32x4{};
                    av = wide(lo, hi);
                } else {
                    av = wide(b + g < blocks ? *reinterpret_cast<const i32x4 *>(a + static_cast<int64_t>(b + g) * 16) : i32x4{});
                }
            }
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(wv[s]), av, acc, kE2M1,
                                                                   FORMAT == SSU_FORMAT_MXFP8 ? kE4M3 : kE2M1, 0, wsv[s], 0, as);
        }
        if constexpr (kFuse) {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }
    sums[wave][l] = acc;
    __syncthreads();
    if (wave == 0) {
        f32x4 v = sums[0][l];
#pragma unroll
        for (int j = 1; j < kStreamWaves; j++)
            v += sums[j][l];
        store_out4<OT>(p, r, n0 + 4 * g, add_bias<OT>(p, n0 + 4 * g, v));
    }
}

// ---------------------------------------------------------------- many rows

// K tile of the tiled kernels: an activation row's tile is 128 bytes in both formats.
template <int FORMAT>
struct KTile {
    static constexpr int kDepth = FORMAT == SSU_FORMAT_MXFP8 ? 128 : 256;
    static constexpr int kSteps = kDepth / 64;  // of the 32x32x64 instruction
    static constexpr int kARow = 128, kWRow = kDepth / 2;  // bytes per row
};
constexpr int ktile_depth(int format) { return format == SSU_FORMAT_MXFP8 ? 128 : 256; }
// K tiles of k values: an even number.
constexpr int64_t ktiles_of(int64_t k, int format) { return (k + 2 * ktile_depth(format) - 1) / (2 * ktile_depth(format)) * 2; }

// Packed scales: for every 32 rows and K tile, 64 words, one per lane of an
// operand (row l % 32, group h = l / 32); byte s is the scale of block STEPS h + s of the tile, 0
// (2^-127) past the end of k. A tile reads its rows' scales without looking where the
// rows end, so there is room for whole tiles; what lies past the last 32 rows
// is not written and goes into sums that are not stored.
__host__ __device__ constexpr int64_t packed_words(int64_t rows, int64_t ktiles) { return (rows + 31) / 32 * ktiles * 64; }
constexpr int64_t packed_room(int64_t rows, int64_t ktiles) { return (rows + 255) / 256 * 8 * ktiles * 64; }

struct PackParams {
    // activations: floats to quantise (codes and packed scales), or codes whose scales are packed
    const void *x;
    const uint8_t *a_scale;
    uint8_t *codes, *a_packed;
    int64_t x_s, as_s;
    // weights' scales
    const uint8_t *w_scale;
    uint32_t *w_packed;
    int64_t ws_s;
    int32_t m, n, k, ktiles;
    int32_t a_groups;  // workgroups that work on the activations; the rest pack the weights' scales
};

template <int FORMAT>
__device__ __forceinline__ void pack_scales(const uint8_t *scale, int64_t stride, int32_t rows, int32_t blocks, int32_t ktiles,
                                            uint32_t *packed, int64_t first, int64_t step) {
    constexpr int kSteps = KTile<FORMAT>::kSteps;
    const int64_t words = packed_words(rows, ktiles);
    for (int64_t i = first; i < words; i += step) {
        const int l = static_cast<int>(i % 64);
        const int64_t t = i / 64;
        const int kt = static_cast<int>(t % ktiles);
        const int64_t row = min(t / ktiles * 32 + l % 32, static_cast<int64_t>(rows) - 1);
        const int b = (2 * kt + l / 32) * kSteps;
        typedef uint32_t Word __attribute__((aligned(1)));
        uint32_t v = 0;
        if (b + 4 <= blocks) {
            v = *reinterpret_cast<const Word *>(scale + row * stride + b);
        } else {
#pragma unroll
            for (int s = 0; s < kSteps; s++)
                if (b + s < blocks)
                    v |= static_cast<uint32_t>(scale[row * stride + b + s]) << (8 * s);
        }
        packed[i] = v;  // of MXFP8 the low half counts
    }
}

// What the tiled kernels need besides the codes: the weights' scales packed,
// and the activations' (quantised here when they come as floats).
template <typename FT, int FORMAT>
__global__ __launch_bounds__(kQuantThreads) void mx_pack_kernel(const PackParams p) {
    constexpr int kSteps = KTile<FORMAT>::kSteps;
    const int blocks = p.k / 32;
    if (static_cast<int>(blockIdx.x) >= p.a_groups) {
        const int64_t at = static_cast<int64_t>(blockIdx.x - p.a_groups) * kQuantThreads + threadIdx.x;
        pack_scales<FORMAT>(p.w_scale, p.ws_s, p.n, blocks, p.ktiles, p.w_packed, at,
                            static_cast<int64_t>(gridDim.x - p.a_groups) * kQuantThreads);
        return;
    }
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(p.a_groups) * kQuantThreads;
    if constexpr (std::is_void_v<FT>) {
        pack_scales<FORMAT>(p.a_scale, p.as_s, p.m, blocks, p.ktiles, reinterpret_cast<uint32_t *>(p.a_packed), first, step);
    } else {
        // four lanes per block of 32, over whole K tiles: the blocks past the end of k get the scale byte 0 and no codes
        const int64_t eighths = static_cast<int64_t>(p.ktiles) * (KTile<FORMAT>::kDepth / 8);
        const int64_t total = p.m * eighths;
        for (int64_t i = first; i < total; i += step) {
            const int64_t row = i / eighths;
            const int at = static_cast<int>(i % eighths) * 8, b = at / 32;
            uint32_t sc = 0;
            if (at < p.k) {
                float v[8];
                load8(static_cast<const FT *>(p.x) + row * p.x_s + at, v);
                uint32_t code[2];
                sc = mx_block<FORMAT>(v, code);
                store_codes<FORMAT>(p.codes + row * (FORMAT == SSU_FORMAT_MXFP4 ? p.k / 2 : p.k), at, code);
            }
            if (i % 4 == 0) {
                const int kt = b / (2 * kSteps), in = b % (2 * kSteps);
                const int64_t word = (row / 32 * p.ktiles + kt) * 64 + in / kSteps * 32 + row % 32;
                p.a_packed[word * 4 + in % kSteps] = static_cast<uint8_t>(sc);
            }
        }
    }
}

struct TileParams {
    MxParams p;
    const uint8_t *a_scales, *w_scales;  // packed words, or rows of scale bytes (p.as_s, p.ws_s)
    int32_t packed;
    int32_t ktiles, mtiles, ntiles;
};

// Byte offset of 16-byte chunk c of row r in an LDS image of rows of 128 or 64 bytes.
// The 64 banks hold two 128-byte lines; a 16-byte read is served for 16 lanes at a time, lanes 0-3,
// 12-15, 20-23 and 24-27 of a half wave together, and these read one chunk of as many rows. With
// the chunks of a line permuted by half its number no two of them share a bank (by its number alone
// every second read collided).
template <int ROW>
__device__ __forceinline__ int lds_chunk(int r, int c) {
    if constexpr (ROW == 128) {
        return r * 128 + ((c ^ ((r >> 1) & 7)) * 16);
    } else {
        const int line = r / 2;
        return line * 128 + ((((r & 1) * 4 + c) ^ ((line >> 1) & 7)) * 16);
    }
}

// Workgroup id to tile: each XCD takes a run of tiles, in groups of eight rows of
// tiles, so that the tiles at work on it share activations and weights in its L2.
__device__ __forceinline__ void tile_at(int id, int mtiles, int ntiles, int *mt, int *nt) {
    const int total = mtiles * ntiles;
    const int per = total / kXcds, rest = total % kXcds, x = id % kXcds;
    const int lin = x * per + min(x, rest) + id / kXcds;
    const int group = lin / (8 * ntiles), first = group * 8, height = min(8, mtiles - first);
    const int in = lin - first * ntiles;
    *mt = first + in % height;
    *nt = in / height;
}

// 16 bytes per lane from memory to 1 KiB of LDS: lane l's bytes go to dst + 16 l.
__device__ __forceinline__ void load_to_lds(const uint8_t *src, uint8_t *dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// Barrier behind which every wave's fills have arrived. The wait is spelled out: the
// compiler's own barrier waits for LDS instructions only, and a wave must not
// pass while what it fetched for the others is on its way.
__device__ __forceinline__ void fills_barrier() {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();
}

// One operand's part in filling an LDS image of ROWS rows of ROW bytes: wave `wave` of
// WAVES loads every WAVES-th KiB. A lane's LDS place is fixed, so the swizzle is in
// which chunk it fetches. Rows past the end fetch the last row; chunks past the end
// of k fetch the row's last chunk, which a scale of 2^-127 on either side takes out of the sum.
template <int ROWS, int ROW, int WAVES>
struct Filler {
    static constexpr int kLoads = ROWS * ROW / 1024 / WAVES;
    static_assert(kLoads * WAVES * 1024 == ROWS * ROW, "whole KiB per wave");
    const uint8_t *row[kLoads];
    int chunk;  // byte offset of this lane's chunk in its row's tile
    int bytes;  // of a row

    __device__ __forceinline__ Filler(const uint8_t *base, int64_t stride, int first, int rows, int row_bytes, int wave, int l) {
        bytes = row_bytes;
        static_assert(WAVES % 2 == 0, "a wave's KiBs are all even ones of the image or all odd ones");
        const int line = l / 8, slot = (l % 8) ^ (wave % 2 * 4 + line / 2);  // as lds_chunk permutes them
        chunk = ROW == 128 ? slot * 16 : slot % 4 * 16;
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int at = (wave + WAVES * i) * 8 + line;
            const int r = ROW == 128 ? at : 2 * at + slot / 4;
            row[i] = base + min(first + r, rows - 1) * stride;
        }
    }
    __device__ __forceinline__ void load(int kt, uint8_t *lds, int wave) const {
        const int64_t at = min(kt * ROW + chunk, bytes - 16);
#pragma unroll
        for (int i = 0; i < kLoads; i++)
            load_to_lds(row[i] + at, lds + (wave + WAVES * i) * 1024);
    }
};

// The end of a tile: sums joined over the waves that split k, bias, rounding and stores, through
// two LDS images of STAGE bytes that are free by now.
template <typename OT, int FM, int FN, int WM, int WN, int WK, int STAGE>
__device__ __forceinline__ void finish_tile(const MxParams &p, f32x16 (&acc)[FM][FN], uint8_t *lds0, uint8_t *lds1, int m0, int n0,
                                            int l, int wave) {
    constexpr int kWaves = WM * WN * WK, kStage = STAGE;
    const int r = l % 32, h = l / 32;
    const int wm = wave % WM, wn = wave / WM % WN, wk = wave / (WM * WN);
    if constexpr (WK > 1) {
        // each wave of the WK that share a part of the tile sums and stores its share of the
        // fragments, half of the registers at a time: the others leave theirs in the LDS images
        static_assert(FM * FN % WK == 0, "fragments divide over the waves");
        constexpr int kShare = FM * FN / WK, kHalf = FM * FN * 8 * 64;  // floats of a wave
        static_assert(WM * WN * WK * kHalf * 4 <= 2 * kStage, "sums fit the images");
        constexpr int kIn0 = kStage / 4 / kHalf;  // waves whose floats go to the first image
        auto sums = [&](int w) {
            return w < kIn0 ? reinterpret_cast<float *>(lds0) + w * kHalf : reinterpret_cast<float *>(lds1) + (w - kIn0) * kHalf;
        };
        const int first = (wn * WM + wm), stride = WM * WN;  // waves first + stride * (0 .. WK - 1) share
        for_passes<0, 2>([&](auto hc) {
            constexpr int half = decltype(hc)::value;
            __syncthreads();
            float *mine = sums(first + stride * wk);
#pragma unroll
            for (int f = 0; f < FM * FN; f++)
                if (f / kShare != wk)
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        mine[(f * 8 + i) * 64 + l] = acc[f / FN][f % FN][half * 8 + i];
            __syncthreads();
#pragma unroll
            for (int f = 0; f < FM * FN; f++) {
                if (f / kShare != wk)
                    continue;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; i++)
                    v[i] = acc[f / FN][f % FN][half * 8 + i];
                for (int o = 1; o < WK; o++) {
                    const float *other = sums(first + stride * ((wk + o) % WK));
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        v[i] += other[(f * 8 + i) * 64 + l];
                }
                const int m = m0 + (wm * FM + f / FN) * 32 + r, n = n0 + (wn * FN + f % FN) * 32 + 4 * h + 16 * half;
                store_out4<OT>(p, m, n, add_bias<OT>(p, n, f32x4{v[0], v[1], v[2], v[3]}));
                store_out4<OT>(p, m, n + 8, add_bias<OT>(p, n + 8, f32x4{v[4], v[5], v[6], v[7]}));
            }
        });
    } else {
        // 32 rows at a time through this wave's part of the images, so that a store writes
        // whole runs of a row: a lane holds four outputs of one row, 32 rows to an instruction
        constexpr int kVec = 16 / static_cast<int>(sizeof(OT)), kCols = 32 * FN;
        constexpr int kLanes = kCols / kVec, kRows = 64 / kLanes;  // lanes per row, rows per store
        constexpr int kRow = kCols + kVec;                         // 16 bytes of padding: rows start on different banks
        static_assert(32 * kRow * static_cast<int>(sizeof(OT)) <= 2 * kStage / kWaves && kWaves % 2 == 0, "slabs fit");
        OT *slab = reinterpret_cast<OT *>((wave % 2 ? lds1 : lds0) + wave / 2 * (2 * kStage / kWaves));
        typedef OT Vec4 __attribute__((ext_vector_type(4)));
        typedef OT VecN __attribute__((ext_vector_type(kVec)));
        typedef OT VecU __attribute__((ext_vector_type(kVec), aligned(sizeof(OT))));
        const int n = n0 + wn * kCols + l % kLanes * kVec;
        for_passes<0, FM>([&](auto ic) {
            constexpr int i = decltype(ic)::value;
#pragma unroll
            for (int j = 0; j < FN; j++)
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    Vec4 v;
                    f32x4 sum = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                    sum = add_bias<OT>(p, n0 + (wn * FN + j) * 32 + 8 * q + 4 * h, sum);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        v[e] = narrow<OT>(sum[e]);
                    *reinterpret_cast<Vec4 *>(slab + r * kRow + j * 32 + 8 * q + 4 * h) = v;
                }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            const int m = m0 + (wm * FM + i) * 32 + l / kLanes;
            const OT *src = slab + l / kLanes * kRow + l % kLanes * kVec;
            OT *dst = static_cast<OT *>(p.out) + m * p.out_s + n;
#pragma unroll
            for (int k = 0; k < 32 / kRows; k++) {
                const VecN v = *reinterpret_cast<const VecN *>(src + k * kRows * kRow);
                if (m + k * kRows < p.m) {
                    OT *at = dst + k * kRows * p.out_s;
                    if (n + kVec <= p.n)
                        *reinterpret_cast<VecU *>(at) = v;
                    else
#pragma unroll
                        for (int e = 0; e < kVec - 1; e++)
                            if (n + e < p.n)
                                at[e] = v[e];
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        });
    }
}

// TM x TN outputs per workgroup; the waves are WM x WN over the tile and WK over the
// steps of a K tile (those join their sums in LDS at the end). Codes go straight
// from memory to two LDS images: while one K tile is multiplied the next arrives. Each
// step's operands are read during the step before, the next tile's first ones
// during this one's last step, behind the only barrier of a tile; the image that
// the tile leaves is filled from there on.
template <typename OT, int FORMAT, int TM, int TN, int WM, int WN, int WK>
__global__ __launch_bounds__(64 * WM * WN * WK) void mx_tile_kernel(const TileParams t) {
    using KT = KTile<FORMAT>;
    constexpr int kWaves = WM * WN * WK;
    constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
    constexpr int kSteps = KT::kSteps / WK;  // of this wave per K tile
    constexpr int kABytes = TM * KT::kARow, kStage = kABytes + TN * KT::kWRow;
    // two arrays, so that the compiler can tell a fill of one from a read of the other
    __shared__ alignas(16) uint8_t lds0[kStage];
    __shared__ alignas(16) uint8_t lds1[kStage];
    const MxParams &p = t.p;
    const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int r = l % 32, h = l / 32;
    const int wm = wave % WM, wn = wave / WM % WN, wk = wave / (WM * WN);
    int mt, nt;
    tile_at(blockIdx.x, t.mtiles, t.ntiles, &mt, &nt);
    const int m0 = mt * TM, n0 = nt * TN;

    const Filler<TM, KT::kARow, kWaves> fill_a(p.a, p.a_s, m0, p.m, FORMAT == SSU_FORMAT_MXFP8 ? p.k : p.k / 2, wave, l);
    const Filler<TN, KT::kWRow, kWaves> fill_w(p.w, p.w_s, n0, p.n, p.k / 2, wave, l);
    auto fill = [&](uint8_t *lds, int kt) {
        fill_a.load(kt, lds, wave);
        fill_w.load(kt, lds + kABytes, wave);
    };
    // scales of this wave's fragments
    const uint32_t *aps = reinterpret_cast<const uint32_t *>(t.a_scales) + (static_cast<int64_t>(m0 / 32 + wm * FM) * t.ktiles) * 64 + l;
    const uint32_t *wps = reinterpret_cast<const uint32_t *>(t.w_scales) + (static_cast<int64_t>(n0 / 32 + wn * FN) * t.ktiles) * 64 + l;
    int asc[FM], wsc[FN], asc_next[FM], wsc_next[FN];
    auto load_scales = [&](int kt) {
#pragma unroll
        for (int i = 0; i < FM; i++)
            asc_next[i] = static_cast<int>(aps[(static_cast<int64_t>(i) * t.ktiles + kt) * 64]);
#pragma unroll
        for (int i = 0; i < FN; i++)
            wsc_next[i] = static_cast<int>(wps[(static_cast<int64_t>(i) * t.ktiles + kt) * 64]);
    };
    struct Frags {
        std::conditional_t<FORMAT == SSU_FORMAT_MXFP8, i32x8, i32x4> a[FM];
        i32x4 w[FN];
    };
    auto read = [&](const uint8_t *src, int j) {
        Frags f;
        const int s = wk + WK * j;
#pragma unroll
        for (int i = 0; i < FM; i++) {
            const int row = (wm * FM + i) * 32 + r;
            if constexpr (FORMAT == SSU_FORMAT_MXFP8)
                f.a[i] = wide(*reinterpret_cast<const i32x4 *>(src + lds_chunk<KT::kARow>(row, 2 * s + h)),
                              *reinterpret_cast<const i32x4 *>(src + lds_chunk<KT::kARow>(row, 2 * (KT::kSteps + s) + h)));
            else
                f.a[i] = *reinterpret_cast<const i32x4 *>(src + lds_chunk<KT::kARow>(row, KT::kSteps * h + s));
        }
#pragma unroll
        for (int i = 0; i < FN; i++)
            f.w[i] = *reinterpret_cast<const i32x4 *>(src + kABytes +
                                                      lds_chunk<KT::kWRow>((wn * FN + i) * 32 + r, KT::kSteps * h + s));
        return f;
    };
    f32x16 acc[FM][FN] = {};
    auto multiply = [&](const Frags &f, auto jc) {
        constexpr int kByte = decltype(jc)::value * WK;
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    wide(f.w[j]), wide(f.a[i]), acc[i][j], kE2M1, FORMAT == SSU_FORMAT_MXFP8 ? kE4M3 : kE2M1, kByte, wsc[j], kByte, asc[i]);
    };

    // k is taken in pairs of tiles without a branch: what lies past its end is
    // filled and multiplied like the rest, and comes to nothing by its scales
    if (t.ktiles > 0) {
        fill(lds0, 0);
        load_scales(0);
        fill(lds1, 1);
        fills_barrier();
        Frags cur = read(lds0, 0);
        auto tile = [&](uint8_t *here, uint8_t *there, int kt) {
#pragma unroll
            for (int i = 0; i < FM; i++)
                asc[i] = WK > 1 ? asc_next[i] >> (8 * wk) : asc_next[i];
#pragma unroll
            for (int i = 0; i < FN; i++)
                wsc[i] = WK > 1 ? wsc_next[i] >> (8 * wk) : wsc_next[i];
            load_scales(min(kt + 1, t.ktiles - 1));
            for_passes<0, kSteps>([&](auto jc) {
                constexpr int j = decltype(jc)::value;
                __builtin_amdgcn_sched_barrier(0);
                Frags next;
                if constexpr (j + 1 < kSteps) {
                    next = read(here, j + 1);
                } else {
                    fills_barrier();
                    next = read(there, 0);
                    fill(here, kt + 2);
                }
                multiply(cur, jc);
                cur = next;
                // the reads (and fills) one by one between the first products
                constexpr int kReads = (FORMAT == SSU_FORMAT_MXFP8 ? 2 * FM : FM) + FN, kFirst = FM * FN > 1 ? FM * FN / 2 : 1;
                constexpr int kFills = j + 1 == kSteps ? decltype(fill_a)::kLoads + decltype(fill_w)::kLoads : 0;
                for_passes<0, kFirst>([&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    __builtin_amdgcn_sched_group_barrier(0x100, kReads * (i + 1) / kFirst - kReads * i / kFirst, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                });
                for_passes<0, FM * FN - kFirst>([&](auto ic) {
                    constexpr int i = decltype(ic)::value, n = FM * FN - kFirst;
                    if constexpr (kFills > 0)
                        __builtin_amdgcn_sched_group_barrier(0x010, kFills * (i + 1) / n - kFills * i / n, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                });
            });
        };
        for (int kt = 0; kt < t.ktiles; kt += 2) {
            tile(lds0, lds1, kt);
            tile(lds1, lds0, kt + 1);
        }
        fills_barrier();
    }

    finish_tile<OT, FM, FN, WM, WN, WK, kStage>(p, acc, lds0, lds1, m0, n0, l, wave);
}

// The smaller tiles: too little work per K tile to hide a fetch behind one of them, so STAGES images
// take turns and a fetch has STAGES - 1 tiles' time. A wave waits for the fetches that the
// next tile needs and no more: only fetches count in vmcnt here (scales come through LDS as well),
// every tile issues the same number of them, and they arrive in order.
template <typename OT, int FORMAT, int TM, int TN, int WM, int WN, int WK, int STAGES>
__global__ __launch_bounds__(64 * WM * WN * WK) void mx_ring_kernel(const TileParams t) {
    using KT = KTile<FORMAT>;
    constexpr int kWaves = WM * WN * WK;
    constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
    constexpr int kSteps = KT::kSteps / WK;
    constexpr int kABytes = TM * KT::kARow, kCodes = kABytes + TN * KT::kWRow;
    constexpr int kScaleTiles = (TM + TN) / 32, kScaleLoads = kScaleTiles / kWaves;  // of 64 words
    constexpr int kStage = kCodes + kScaleTiles * 256;
    static_assert(kScaleLoads * kWaves == kScaleTiles, "whole words per wave");
    static_assert(STAGES == 4 || STAGES == 8, "images");
    // arrays of their own: the compiler tells fills of one from reads of another
    __shared__ alignas(16) uint8_t s0[kStage], s1[kStage], s2[kStage], s3[kStage];
    __shared__ alignas(16) uint8_t s4[STAGES > 4 ? kStage : 16], s5[STAGES > 4 ? kStage : 16], s6[STAGES > 4 ? kStage : 16],
        s7[STAGES > 4 ? kStage : 16];
    const MxParams &p = t.p;
    const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int r = l % 32, h = l / 32;
    const int wm = wave % WM, wn = wave / WM % WN, wk = wave / (WM * WN);
    int mt, nt;
    tile_at(blockIdx.x, t.mtiles, t.ntiles, &mt, &nt);
    const int m0 = mt * TM, n0 = nt * TN;

    const Filler<TM, KT::kARow, kWaves> fill_a(p.a, p.a_s, m0, p.m, FORMAT == SSU_FORMAT_MXFP8 ? p.k : p.k / 2, wave, l);
    const Filler<TN, KT::kWRow, kWaves> fill_w(p.w, p.w_s, n0, p.n, p.k / 2, wave, l);
    // scale words: packed, or straight from rows of bytes (a word of MXFP4's is the four of
    // half h, of MXFP8's the four of the tile)
    const uint8_t *scale[kScaleLoads];
#pragma unroll
    for (int i = 0; i < kScaleLoads; i++) {
        const int tile = wave + kWaves * i;
        const bool is_a = tile < TM / 32;
        const int row0 = is_a ? m0 + tile * 32 : n0 + (tile - TM / 32) * 32;
        const uint8_t *base = is_a ? t.a_scales : t.w_scales;
        if (t.packed)
            scale[i] = base + (static_cast<int64_t>(row0 / 32) * t.ktiles * 64 + l) * 4;
        else
            scale[i] = base + static_cast<int64_t>(min(row0 + r, (is_a ? p.m : p.n) - 1)) * (is_a ? p.as_s : p.ws_s) +
                       (FORMAT == SSU_FORMAT_MXFP8 ? 0 : 4 * h);
    }
    const int scale_step = t.packed ? 256 : KT::kDepth / 32;
    const int shift = 8 * wk + (FORMAT == SSU_FORMAT_MXFP8 && !t.packed ? 16 * h : 0);
    constexpr int kLoads = decltype(fill_a)::kLoads + decltype(fill_w)::kLoads + kScaleLoads;
    auto fill = [&](uint8_t *lds, int kt) {
        fill_a.load(kt, lds, wave);
        fill_w.load(kt, lds + kABytes, wave);
        const int64_t at = static_cast<int64_t>(min(kt, t.ktiles - 1)) * scale_step;
#pragma unroll
        for (int i = 0; i < kScaleLoads; i++)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)(scale[i] + at),
                (__attribute__((address_space(3))) void *)(lds + kCodes + (wave + kWaves * i) * 256), 4, 0, 0);
    };
    struct Frags {
        std::conditional_t<FORMAT == SSU_FORMAT_MXFP8, i32x8, i32x4> a[FM];
        i32x4 w[FN];
    };
    auto read = [&](const uint8_t *src, int j) {
        Frags f;
        const int s = wk + WK * j;
#pragma unroll
        for (int i = 0; i < FM; i++) {
            const int row = (wm * FM + i) * 32 + r;
            if constexpr (FORMAT == SSU_FORMAT_MXFP8)
                f.a[i] = wide(*reinterpret_cast<const i32x4 *>(src + lds_chunk<KT::kARow>(row, 2 * s + h)),
                              *reinterpret_cast<const i32x4 *>(src + lds_chunk<KT::kARow>(row, 2 * (KT::kSteps + s) + h)));
            else
                f.a[i] = *reinterpret_cast<const i32x4 *>(src + lds_chunk<KT::kARow>(row, KT::kSteps * h + s));
        }
#pragma unroll
        for (int i = 0; i < FN; i++)
            f.w[i] = *reinterpret_cast<const i32x4 *>(src + kABytes +
                                                      lds_chunk<KT::kWRow>((wn * FN + i) * 32 + r, KT::kSteps * h + s));
        return f;
    };
    int asc[FM], wsc[FN];
    auto read_scales = [&](const uint8_t *src) {
        const uint32_t *words = reinterpret_cast<const uint32_t *>(src + kCodes) + l;
#pragma unroll
        for (int i = 0; i < FM; i++)
            asc[i] = static_cast<int>(words[(wm * FM + i) * 64]);
#pragma unroll
        for (int i = 0; i < FN; i++)
            wsc[i] = static_cast<int>(words[(TM / 32 + wn * FN + i) * 64]);
    };
    f32x16 acc[FM][FN] = {};
    auto multiply = [&](const Frags &f, auto jc) {
        constexpr int kByte = decltype(jc)::value * WK;
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    wide(f.w[j]), wide(f.a[i]), acc[i][j], kE2M1, FORMAT == SSU_FORMAT_MXFP8 ? kE4M3 : kE2M1, kByte, wsc[j], kByte, asc[i]);
    };
    // waits until at most `pending` fetches of this wave are outstanding (and no LDS access, if
    // `lds`), then for the other waves
    auto arrive = [](auto pending, auto lds) {
        constexpr int n = decltype(pending)::value;
        static_assert(n < 64, "vmcnt has six bits");
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((decltype(lds)::value ? 0x0070 : 0x0F70) | (n & 15) | ((n >> 4) << 14));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    uint8_t *const images[8] = {s0, s1, s2, s3, s4, s5, s6, s7};
    if (t.ktiles > 0) {
        for_passes<0, STAGES>([&](auto sc) { fill(images[decltype(sc)::value], decltype(sc)::value); });
        if constexpr (kSteps == 1) {
            // A wave has one step per K tile: its operands are read two tiles ahead, so that neither
            // the fetch nor the LDS is waited for. When a wave arrives, it has multiplied tile
            // kt, so its reads of that image are complete and the image can be filled.
            arrive(std::integral_constant<int, (STAGES - 2) * kLoads>(), std::true_type());
            Frags cur = read(s0, 0), next = read(s1, 0);
            int a0[FM], w0[FN], a1[FM], w1[FN];
            auto words = [&](const uint8_t *src, int (&a)[FM], int (&w)[FN]) {
                read_scales(src);
#pragma unroll
                for (int i = 0; i < FM; i++)
                    a[i] = asc[i];
#pragma unroll
                for (int i = 0; i < FN; i++)
                    w[i] = wsc[i];
            };
            words(s0, a0, w0);
            words(s1, a1, w1);
            int kt = 0;
            bool done = false;
            while (!done) {
                for_passes<0, STAGES>([&](auto sc) {
                    constexpr int s = decltype(sc)::value;
                    if (done)
                        return;
#pragma unroll
                    for (int i = 0; i < FM; i++)
                        asc[i] = a0[i] >> shift;
#pragma unroll
                    for (int i = 0; i < FN; i++)
                        wsc[i] = w0[i] >> shift;
                    multiply(cur, std::integral_constant<int, 0>());
                    __builtin_amdgcn_sched_barrier(0);
                    arrive(std::integral_constant<int, (STAGES - 3) * kLoads>(), std::false_type());
                    cur = next;
#pragma unroll
                    for (int i = 0; i < FM; i++)
                        a0[i] = a1[i];
#pragma unroll
                    for (int i = 0; i < FN; i++)
                        w0[i] = w1[i];
                    next = read(images[(s + 2) % STAGES], 0);
                    words(images[(s + 2) % STAGES], a1, w1);
                    __builtin_amdgcn_sched_barrier(0);
                    fill(images[s], kt + STAGES);
                    done = ++kt >= t.ktiles;
                });
            }
        } else {
            arrive(std::integral_constant<int, (STAGES - 1) * kLoads>(), std::true_type());
            Frags cur = read(s0, 0);
            auto shifted_scales = [&](const uint8_t *src) {
                read_scales(src);
#pragma unroll
                for (int i = 0; i < FM; i++)
                    asc[i] >>= shift;
#pragma unroll
                for (int i = 0; i < FN; i++)
                    wsc[i] >>= shift;
            };
            shifted_scales(s0);
            auto tile = [&](uint8_t *here, uint8_t *there, int kt) {
                for_passes<0, kSteps>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    Frags next;
                    if constexpr (j + 1 < kSteps) {
                        next = read(here, j + 1);
                        multiply(cur, jc);
                    } else {
                        // the products first: they need nothing that is still on its way
                        multiply(cur, jc);
                        arrive(std::integral_constant<int, (STAGES - 2) * kLoads>(), std::true_type());
                        next = read(there, 0);
                        shifted_scales(there);
                        fill(here, kt + STAGES);
                    }
                    cur = next;
                });
            };
            int kt = 0;
            bool done = false;
            while (!done) {
                for_passes<0, STAGES>([&](auto sc) {
                    constexpr int s = decltype(sc)::value;
                    if (done)
                        return;
                    tile(images[s], images[(s + 1) % STAGES], kt);
                    done = ++kt >= t.ktiles;
                });
            }
        }
        arrive(std::integral_constant<int, 0>(), std::true_type());  // the last fills and reads
    }
    finish_tile<OT, FM, FN, WM, WN, WK, kStage>(p, acc, s0, s1, m0, n0, l, wave);
}

// ---------------------------------------------------------------- launches

template <typename T>
const void *quantize_fn(int format) {
    return format == SSU_FORMAT_MXFP4 ? reinterpret_cast<const void *>(&mx_quantize_rows_kernel<T, SSU_FORMAT_MXFP4>)
                                      : reinterpret_cast<const void *>(&mx_quantize_rows_kernel<T, SSU_FORMAT_MXFP8>);
}
template <typename FT>
const void *pack_fn(int format) {
    return format == SSU_FORMAT_MXFP4 ? reinterpret_cast<const void *>(&mx_pack_kernel<FT, SSU_FORMAT_MXFP4>)
                                      : reinterpret_cast<const void *>(&mx_pack_kernel<FT, SSU_FORMAT_MXFP8>);
}
template <typename OT, int FORMAT>
const void *stream_fn(bool fuse, int x_dtype) {
    if (fuse)
        return x_dtype == SSU_F32   ? reinterpret_cast<const void *>(&mx_stream_kernel<OT, FORMAT, float>)
               : x_dtype == SSU_F16 ? reinterpret_cast<const void *>(&mx_stream_kernel<OT, FORMAT, _Float16>)
                                    : reinterpret_cast<const void *>(&mx_stream_kernel<OT, FORMAT, __bf16>);
    return reinterpret_cast<const void *>(&mx_stream_kernel<OT, FORMAT, void>);
}

struct TileShape {
    int tm, tn;
};
constexpr TileShape kTileShapes[4] = {{256, 256}, {128, 128}, {64, 64}, {64, 64}};
constexpr int kTileThreads = 256;

template <typename OT, int FORMAT>
const void *tile_fn(int shape) {
    constexpr int kWk = KTile<FORMAT>::kSteps;
    switch (shape) {
    case 0: return reinterpret_cast<const void *>(&mx_tile_kernel<OT, FORMAT, 256, 256, 2, 2, 1>);
    case 1: return reinterpret_cast<const void *>(&mx_ring_kernel<OT, FORMAT, 128, 128, 2, 2, 1, 4>);
    case 2: return reinterpret_cast<const void *>(&mx_ring_kernel<OT, FORMAT, 64, 64, 1, 4 / kWk, kWk, 4>);
    }
    return reinterpret_cast<const void *>(&mx_ring_kernel<OT, FORMAT, 64, 64, 1, 4 / kWk, kWk, 8>);
}

// The largest tile that leaves every compute unit one; of the smallest, the form with eight
// images if no unit gets a second one, else the one with four, of which two fit a unit.
int tile_shape(int64_t m, int64_t n) {
    for (int s = 0; s < 3; s++)
        if (((m + kTileShapes[s].tm - 1) / kTileShapes[s].tm) * ((n + kTileShapes[s].tn - 1) / kTileShapes[s].tn) >= (s < 2 ? 256 : 257))
            return s;
    return 3;
}
// Whether a tile's scale words can be fetched where the bytes are: the large tile packs them first (it
// would fetch a line for eight bytes of each of 512 rows), and so do words that are not aligned or
// reach past the end of k.
bool scales_in_place(int shape, const void *base, int64_t stride, int64_t k, int format) {
    return shape != 0 && k % ktile_depth(format) == 0 && stride % 4 == 0 && reinterpret_cast<uintptr_t>(base) % 4 == 0;
}

template <typename F>
const void *by_out(int out_dtype, F &&f) {
    return out_dtype == SSU_F32 ? f(0.0f) : out_dtype == SSU_F16 ? f(static_cast<_Float16>(0)) : f(static_cast<__bf16>(0));
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t code_bytes(int64_t m, int64_t k, int format) { return round256(format == SSU_FORMAT_MXFP4 ? m * k / 2 : m * k); }

int run(const void *fn, int64_t grid, int block, void **args, void *stream) {
    if (grid > INT32_MAX)
        return static_cast<int>(hipErrorInvalidValue);
    return static_cast<int>(hipLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(block), args, 0,
                                            static_cast<hipStream_t>(stream)));
}

}  // namespace

int launch_mx_quantize_rows(const void *src, int dtype, int64_t stride, int64_t rows, int64_t k, uint8_t *codes,
                            uint8_t *scales, int format, void *stream) {
    const void *fn = dtype == SSU_F32   ? quantize_fn<float>(format)
                     : dtype == SSU_F16 ? quantize_fn<_Float16>(format)
                                        : quantize_fn<__bf16>(format);
    int64_t blocks = (rows * (k / 8) + kQuantThreads - 1) / kQuantThreads;
    blocks = blocks > 65536 ? 65536 : blocks;
    int32_t k32 = static_cast<int32_t>(k);
    void *args[] = {&src, &stride, &rows, &k32, &codes, &scales};
    return run(fn, blocks, kQuantThreads, args, stream);
}

int64_t mx_linear_workspace(int64_t m, int64_t n, int64_t k, int format, bool floats) {
    const int64_t quantised = floats && m > kMxFuseRows ? code_bytes(m, k, format) + round256(m * (k / 32)) : 0;
    if (m <= kMxRowsMax)
        return quantised;
    const int64_t ktiles = ktiles_of(k, format);
    return quantised + 4 * (packed_room(m, ktiles) + packed_room(n, ktiles));
}

int launch_mx_linear(const MxParams &args_in, int format, int out_dtype, void *stream) {
    MxParams p = args_in;
    const bool mx4 = format == SSU_FORMAT_MXFP4;
    const bool floats = p.x != nullptr;
    uint8_t *ws = p.workspace;
    const bool fuse = floats && p.m <= kMxFuseRows;
    const int shape = tile_shape(p.m, p.n);
    // where scales are packed, the activations are quantised in the same launch
    const bool packs_floats = floats && p.m > kMxRowsMax && !scales_in_place(shape, p.w_scale, p.ws_s, p.k, format);
    if (floats && !fuse && !packs_floats && p.k > 0) {
        uint8_t *scales = ws + code_bytes(p.m, p.k, format);
        if (int e = launch_mx_quantize_rows(p.x, p.x_dtype, p.x_s, p.m, p.k, ws, scales, format, stream))
            return e;
        p.a = ws;
        p.a_scale = scales;
        p.a_s = mx4 ? p.k / 2 : p.k;
        p.as_s = p.k / 32;
    }
    if (floats && !fuse)
        ws += code_bytes(p.m, p.k, format) + round256(static_cast<int64_t>(p.m) * (p.k / 32));
    if (p.m <= kMxRowsMax) {
        const void *fn = by_out(out_dtype, [&](auto o) {
            using OT = decltype(o);
            return mx4 ? stream_fn<OT, SSU_FORMAT_MXFP4>(fuse, p.x_dtype) : stream_fn<OT, SSU_FORMAT_MXFP8>(fuse, p.x_dtype);
        });
        void *args[] = {&p};
        return run(fn, (p.n + kStreamRows - 1) / kStreamRows, kStreamWaves * 64, args, stream);
    }

    TileParams t = {};
    t.packed = packs_floats || !scales_in_place(shape, p.a_scale, p.as_s, p.k, format) ||
               !scales_in_place(shape, p.w_scale, p.ws_s, p.k, format);
    t.ktiles = static_cast<int32_t>(t.packed ? ktiles_of(p.k, format) : p.k / ktile_depth(format));
    t.a_scales = p.a_scale;
    t.w_scales = p.w_scale;
    if (t.packed && t.ktiles > 0) {
        PackParams q = {};
        if (packs_floats) {
            q.x = p.x;
            q.x_s = p.x_s;
            q.codes = p.workspace;
            p.a = p.workspace;
            p.a_s = mx4 ? p.k / 2 : p.k;
        } else {
            q.a_scale = p.a_scale;
            q.as_s = p.as_s;
        }
        q.a_packed = ws;
        q.w_packed = reinterpret_cast<uint32_t *>(ws) + packed_room(p.m, t.ktiles);
        q.w_scale = p.w_scale;
        q.ws_s = p.ws_s;
        q.m = p.m, q.n = p.n, q.k = p.k, q.ktiles = t.ktiles;
        const int64_t a_work = packs_floats ? static_cast<int64_t>(p.m) * t.ktiles * (ktile_depth(format) / 8) : packed_words(p.m, t.ktiles);
        const int64_t w_work = packed_words(p.n, t.ktiles);
        const auto groups = [](int64_t work) { return static_cast<int>(std::min<int64_t>((work + kQuantThreads - 1) / kQuantThreads, 32768)); };
        q.a_groups = groups(a_work);
        const void *fn = !packs_floats          ? pack_fn<void>(format)
                         : p.x_dtype == SSU_F32 ? pack_fn<float>(format)
                         : p.x_dtype == SSU_F16 ? pack_fn<_Float16>(format)
                                                : pack_fn<__bf16>(format);
        void *args[] = {&q};
        if (int e = run(fn, q.a_groups + groups(w_work), kQuantThreads, args, stream))
            return e;
        t.a_scales = q.a_packed;
        t.w_scales = reinterpret_cast<const uint8_t *>(q.w_packed);
    }
    t.p = p;
    t.mtiles = (p.m + kTileShapes[shape].tm - 1) / kTileShapes[shape].tm;
    t.ntiles = (p.n + kTileShapes[shape].tn - 1) / kTileShapes[shape].tn;
    const void *fn = by_out(out_dtype, [&](auto o) {
        using OT = decltype(o);
        return mx4 ? tile_fn<OT, SSU_FORMAT_MXFP4>(shape) : tile_fn<OT, SSU_FORMAT_MXFP8>(shape);
    });
    void *args[] = {&t};
    return run(fn, static_cast<int64_t>(t.mtiles) * t.ntiles, kTileThreads, args, stream);
}

}  // namespace ssu
