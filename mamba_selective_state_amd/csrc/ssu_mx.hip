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
// k and join their sums in LDS (by the waves' order, so that results repeat). 16 outputs, the
// least of an instruction, give the most workgroups: 18560 x 4096 weights, one bf16 row quantised to
// MXFP8 on the way, take 8.7 us (40.4 MB, 4.6 TB/s).
//
// kMxRowsMax: with 16 rows 18560 x 4096 MXFP8 takes 20.9 us here and 21.7 in the tiled kernels, with 32 34.6
// and 23.4; 4096 x 8192 MXFP4 10.2 and 14.9, 13.4 and 15.8: there 32 rows too would be faster here, which a rule by rows
// alone gives away. 16 is also the instruction's other side.
// kMxFuseRows: every workgroup quantises all rows for itself: 12.4 us with 4 rows, where a
// launch of its own takes 15.8 for 5; the work grows with the rows, and the LDS for them.

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
            wave_lds_fence();
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
            wave_lds_fence();
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

// Scales for the large tile, packed: for every 32 rows and K tile, 64 words, one per lane of
// an operand (row l % 32, group h = l / 32); byte s is the scale of block STEPS h + s of the tile, 0
// (2^-127) past the end of k. A tile reads its rows' scales without looking where the
// rows end, so there is room for whole tiles; what lies past the last 32 rows
// is not written and goes into sums that are not stored.
__host__ __device__ constexpr int64_t packed_words(int64_t rows, int64_t ktiles) { return (rows + 31) / 32 * ktiles * 64; }
constexpr int64_t packed_room(int64_t rows, int64_t ktiles) { return (rows + 255) / 256 * 8 * ktiles * 64; }
// Scales for the smaller tiles: rows of bytes as they are, if they consist of aligned runs of 16
// (k a multiple of 512); else copied to such rows, with 0 past the end of k.
__host__ __device__ constexpr int64_t padded_scales(int64_t k) { return (k + 511) / 512 * 16; }

struct PackParams {
    // activations: floats to quantise, or scale bytes to lay out
    const void *x;
    const uint8_t *a_scale;
    uint8_t *codes, *a_out;
    int64_t x_s, as_s;
    // weights' scales
    const uint8_t *w_scale;
    uint8_t *w_out;
    int64_t ws_s;
    int32_t m, n, k;
    int32_t ktiles;    // even; 0: padded rows
    int32_t a_groups;  // workgroups that work on the activations; the rest lay out the weights' scales
};

template <int FORMAT>
__device__ __forceinline__ void lay_out_scales(const uint8_t *scale, int64_t stride, int32_t rows, int32_t k, int32_t ktiles,
                                               uint8_t *out, int64_t first, int64_t step) {
    constexpr int kSteps = KTile<FORMAT>::kSteps;
    typedef uint32_t Word __attribute__((aligned(1)));
    const int blocks = k / 32;
    // the four bytes of a row from block b on
    auto word = [&](int64_t row, int b, int want) {
        if (b + 4 <= blocks)
            return static_cast<uint32_t>(*reinterpret_cast<const Word *>(scale + row * stride + b));
        uint32_t v = 0;
        for (int s = 0; s < want; s++)
            if (b + s < blocks)
                v |= static_cast<uint32_t>(scale[row * stride + b + s]) << (8 * s);
        return v;
    };
    uint32_t *words = reinterpret_cast<uint32_t *>(out);
    if (ktiles > 0) {
        const int64_t total = packed_words(rows, ktiles);
        for (int64_t i = first; i < total; i += step) {
            const int l = static_cast<int>(i % 64);
            const int64_t t = i / 64;
            const int kt = static_cast<int>(t % ktiles);
            const int64_t row = min(t / ktiles * 32 + l % 32, static_cast<int64_t>(rows) - 1);
            words[i] = word(row, (2 * kt + l / 32) * kSteps, kSteps);  // of MXFP8 the low half counts
        }
    } else {
        const int64_t per = padded_scales(k) / 4;
        for (int64_t i = first; i < rows * per; i += step)
            words[i] = word(i / per, static_cast<int>(i % per) * 4, 4);
    }
}

// What the tiled kernels need besides the codes: scales laid out, and activations that come as
// floats quantised.
template <typename FT, int FORMAT>
__global__ __launch_bounds__(kQuantThreads) void mx_pack_kernel(const PackParams p) {
    constexpr int kSteps = KTile<FORMAT>::kSteps;
    if (static_cast<int>(blockIdx.x) >= p.a_groups) {
        const int64_t at = static_cast<int64_t>(blockIdx.x - p.a_groups) * kQuantThreads + threadIdx.x;
        lay_out_scales<FORMAT>(p.w_scale, p.ws_s, p.n, p.k, p.ktiles, p.w_out, at,
                               static_cast<int64_t>(gridDim.x - p.a_groups) * kQuantThreads);
        return;
    }
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kQuantThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(p.a_groups) * kQuantThreads;
    if constexpr (std::is_void_v<FT>) {
        lay_out_scales<FORMAT>(p.a_scale, p.as_s, p.m, p.k, p.ktiles, p.a_out, first, step);
    } else {
        // four lanes per block of 32, over whole K tiles (or padded rows): the blocks past the end of k
        // get the scale byte 0 and no codes
        const int64_t row_scales = p.ktiles > 0 ? static_cast<int64_t>(p.ktiles) * (KTile<FORMAT>::kDepth / 32) : padded_scales(p.k);
        const int64_t eighths = row_scales * 4;
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
                int64_t to = row * row_scales + b;
                if (p.ktiles > 0) {
                    const int kt = b / (2 * kSteps), in = b % (2 * kSteps);
                    to = ((row / 32 * p.ktiles + kt) * 64 + in / kSteps * 32 + row % 32) * 4 + in % kSteps;
                }
                p.a_out[to] = static_cast<uint8_t>(sc);
            }
        }
    }
}

struct TileParams {
    MxParams p;
    const uint8_t *a_scales, *w_scales;  // packed words, or rows of scale bytes (p.as_s, p.ws_s: multiples of 16)
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
            wave_lds_fence();
            const int m = m0 + (wm * FM + i) * 32 + l / kLanes;
            const OT *src = slab + l / kLanes * kRow + l % kLanes * kVec;
            OT *dst = static_cast<OT *>(p.out) + m * p.out_s + n;
#pragma unroll
            for (int k = 0; k < 32 / kRows; k++) {
                const VecN v = *reinterpret_cast<const VecN *>(src + k * kRows * kRow);
                if (m + k * kRows < p.m) {
                    OT *at = dst + k * kRows * p.out_s;
                    if (n + kVec <= p.n)
                        __builtin_nontemporal_store(static_cast<VecU>(v), reinterpret_cast<VecU *>(at));
                    else
#pragma unroll
                        for (int e = 0; e < kVec - 1; e++)
                            if (n + e < p.n)
                                at[e] = v[e];
                }
            }
            wave_lds_fence();
        });
    }
}

// The matrix instructions bound it, and the 64 KB per K tile that come from the L2: 8192 x 18560 x 4096 MXFP4
// runs at 3300 TF in all (375 us with the 20 of the quantisation; 367 to 387 from run to run). By the
// kernel's times with 8192 x 18432 (nine rounds of tiles) from k = 1024 to 8192, 139 to 600 us, the loop
// runs at 4700 TF (MXFP8, 175 to 888 us: 3000), where registers alone reach 6800 (5200 with zero codes, which draw less
// power), and 8 us a round do not depend on k (12 with 8192 x 8192, four rounds): a tile's first fetches and its
// stores, which no other workgroup covers. A wave has all 512 registers of its lanes, half of them sums,
// so a compute unit holds one workgroup. Four images or more outputs per wave brought nothing. The stores of whole
// runs go past the caches, which keep activations and weights (408 us without, 388 with them then).
//
// TM x TN outputs per workgroup; the waves are WM x WN over the tile. Codes go straight
// from memory to two LDS images: while one K tile is multiplied the next arrives. Each
// step's operands are read during the step before, the next tile's first ones
// during this one's last step, behind the only barrier of a tile; the image that
// the tile leaves is filled from there on.
template <typename OT, int FORMAT, int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void mx_tile_kernel(const TileParams t) {
    using KT = KTile<FORMAT>;
    constexpr int kWaves = WM * WN;
    constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
    constexpr int kSteps = KT::kSteps;
    constexpr int kABytes = TM * KT::kARow, kStage = kABytes + TN * KT::kWRow;
    // two arrays, so that the compiler can tell a fill of one from a read of the other
    __shared__ alignas(16) uint8_t lds0[kStage];
    __shared__ alignas(16) uint8_t lds1[kStage];
    const MxParams &p = t.p;
    const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int r = l % 32, h = l / 32;
    const int wm = wave % WM, wn = wave / WM;
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
    auto read = [&](const uint8_t *src, int s) {
        Frags f;
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
        constexpr int kByte = decltype(jc)::value;
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
                asc[i] = asc_next[i];
#pragma unroll
            for (int i = 0; i < FN; i++)
                wsc[i] = wsc_next[i];
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

    finish_tile<OT, FM, FN, WM, WN, 1, kStage>(p, acc, lds0, lds1, m0, n0, l, wave);
}

// 256 x 4096 x 8192 MXFP4: 14.6 us (24 MB at 1.6 TB/s from HBM, but every workgroup reads
// 0.8 MB from the L2; its fetches' way, 32 K tiles one after another, bounds it).
//
// The smaller tiles: too little work per K tile to hide a fetch behind one of them, so four images
// of SUB K tiles take turns. A wave waits for the fetches that the next products need and no
// more: only fetches count in vmcnt here, every image issues the same number of them, and they
// arrive in order. The scale bytes of four images (a round) come together, 16 bytes of a row at a time, into
// one of two places: a word for each lane and K tile took as long as all the codes.
template <typename OT, int FORMAT, int TM, int TN, int WM, int WN, int WK, int SUB>
__global__ __launch_bounds__(64 * WM * WN * WK) void mx_ring_kernel(const TileParams t) {
    using KT = KTile<FORMAT>;
    constexpr int kWaves = WM * WN * WK;
    constexpr int FM = TM / WM / 32, FN = TN / WN / 32;
    constexpr int kSteps = KT::kSteps / WK;
    constexpr int kImages = 4;
    constexpr int kABytes = TM * KT::kARow, kOne = kABytes + TN * KT::kWRow, kStage = SUB * kOne;  // of a K tile, of an image
    // scale bytes of a round: kRuns runs of 16 per row, the runs permuted so that 16 neighbouring rows'
    // words lie on different banks
    constexpr int kRoundK = kImages * SUB * KT::kDepth;
    constexpr int kRuns = kRoundK / 512, kScaleRow = 16 * kRuns;
    constexpr int kScaleKiB = (TM + TN) * kScaleRow / 1024;
    constexpr int kScaleLoads = kScaleKiB > kWaves ? kScaleKiB / kWaves : 1;
    static_assert(kRuns <= 2, "one bit of the row permutes them");
    static_assert(kScaleKiB % kWaves == 0 || kWaves % kScaleKiB == 0, "every wave fetches as many");
    static_assert(SUB == 1 || kSteps == 1, "images of several K tiles are for one step per tile");
    // arrays of their own: the compiler tells fills of one from reads of another
    __shared__ alignas(16) uint8_t s0[kStage], s1[kStage], s2[kStage], s3[kStage];
    __shared__ alignas(16) uint8_t c0[(TM + TN) * kScaleRow], c1[(TM + TN) * kScaleRow];
    const MxParams &p = t.p;
    const int l = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int r = l % 32, h = l / 32;
    const int wm = wave % WM, wn = wave / WM % WN, wk = wave / (WM * WN);
    int mt, nt;
    tile_at(blockIdx.x, t.mtiles, t.ntiles, &mt, &nt);
    const int m0 = mt * TM, n0 = nt * TN;

    const Filler<TM, KT::kARow, kWaves> fill_a(p.a, p.a_s, m0, p.m, FORMAT == SSU_FORMAT_MXFP8 ? p.k : p.k / 2, wave, l);
    const Filler<TN, KT::kWRow, kWaves> fill_w(p.w, p.w_s, n0, p.n, p.k / 2, wave, l);
    constexpr int kLoads = SUB * (decltype(fill_a)::kLoads + decltype(fill_w)::kLoads);
    // the waits count fetches in the order in which they are written down here
    auto in_order = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // image number `n` of the sequence
    auto fill = [&](uint8_t *lds, int n) {
        in_order();
#pragma unroll
        for (int u = 0; u < SUB; u++) {
            fill_a.load(n * SUB + u, lds + u * kOne, wave);
            fill_w.load(n * SUB + u, lds + u * kOne + kABytes, wave);
        }
        in_order();
    };
    auto permuted = [](int row, int run) { return kRuns == 2 ? run ^ ((row >> 3) & 1) : run; };
    const uint8_t *scale[kScaleLoads];
    int scale_at[kScaleLoads];
#pragma unroll
    for (int i = 0; i < kScaleLoads; i++) {
        const int unit = (wave + kWaves * i) % kScaleKiB * 64 + l, row = unit / kRuns;  // waves too many fetch the same again
        const bool is_a = row < TM;
        scale[i] = is_a ? t.a_scales + min(m0 + row, p.m - 1) * p.as_s : t.w_scales + min(n0 + row - TM, p.n - 1) * p.ws_s;
        scale_at[i] = permuted(row, unit % kRuns) * 16;
    }
    const int scale_last = t.ktiles * (KT::kDepth / 32) - 16;
    // the scales of round `n`; past the end the last run
    auto fill_scales = [&](uint8_t *lds, int n) {
#pragma unroll
        for (int i = 0; i < kScaleLoads; i++)
            load_to_lds(scale[i] + min(n * kScaleRow + scale_at[i], scale_last), lds + (wave + kWaves * i) % kScaleKiB * 1024);
        in_order();
    };
    struct Operands {
        std::conditional_t<FORMAT == SSU_FORMAT_MXFP8, i32x8, i32x4> a[FM];
        i32x4 w[FN];
    };
    // operands of this wave's step `j` of the K tile at `src`
    auto read = [&](const uint8_t *src, int j) {
        Operands f;
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
    // Words with the scales of K tile `kt` of a round: of MXFP4 the four bytes of half h, of
    // MXFP8 all four, of which the half is the upper or the lower two.
    struct Scales {
        uint32_t a[FM], w[FN];
    };
    constexpr int kWord = FORMAT == SSU_FORMAT_MXFP8 ? 4 : 8;  // bytes of a row per K tile
    auto read_scales = [&](const uint8_t *src, int kt) {
        Scales f;
        auto word = [&](int row) {
            const int byte = kt * kWord + (FORMAT == SSU_FORMAT_MXFP8 ? 0 : 4 * h);
            return *reinterpret_cast<const uint32_t *>(src + row * kScaleRow + permuted(row, byte / 16) * 16 + byte % 16);
        };
#pragma unroll
        for (int i = 0; i < FM; i++)
            f.a[i] = word((wm * FM + i) * 32 + r);
#pragma unroll
        for (int i = 0; i < FN; i++)
            f.w[i] = word(TM + (wn * FN + i) * 32 + r);
        return f;
    };
    const int shift = 8 * wk + (FORMAT == SSU_FORMAT_MXFP8 ? 16 * h : 0);
    f32x16 acc[FM][FN] = {};
    auto multiply = [&](const Operands &f, const Scales &sc, auto jc) {
        constexpr int kByte = decltype(jc)::value * WK;
        int as[FM], ws[FN];
#pragma unroll
        for (int i = 0; i < FM; i++)
            as[i] = static_cast<int>(sc.a[i] >> shift);
#pragma unroll
        for (int i = 0; i < FN; i++)
            ws[i] = static_cast<int>(sc.w[i] >> shift);
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    wide(f.w[j]), wide(f.a[i]), acc[i][j], kE2M1, FORMAT == SSU_FORMAT_MXFP8 ? kE4M3 : kE2M1, kByte, ws[j], kByte, as[i]);
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
    uint8_t *const images[kImages] = {s0, s1, s2, s3};
    uint8_t *const places[2] = {c0, c1};
    const int all = t.ktiles / SUB;
    if (all > 0) {
        int n = 0;
        bool done = false;
        if constexpr (kSteps == 1) {
            // A wave has one step per K tile: its operands are read two images ahead, so that neither
            // the fetch nor the LDS is waited for. When the waves have arrived, all have multiplied image
            // n, so their reads of it, and of the scales up to its own, are complete: it can be filled
            // again, and behind a round's last image the place of its scales. In order of issue:
            // image 4 i + 3, scales of round i + 1, image 4 i + 4, ...
            fill_scales(c0, 0);
            fill(s0, 0);
            fill(s1, 1);
            fill(s2, 2);
            fill(s3, 3);
            fill_scales(c1, 1);
            arrive(std::integral_constant<int, 2 * kLoads + kScaleLoads>(), std::true_type());
            struct Image {
                Operands f[SUB];
                Scales s[SUB];
            };
            auto read_all = [&](const uint8_t *src, const uint8_t *scales, int i) {
                Image o;
#pragma unroll
                for (int u = 0; u < SUB; u++) {
                    o.f[u] = read(src + u * kOne, 0);
                    o.s[u] = read_scales(scales, i * SUB + u);
                }
                return o;
            };
            Image cur = read_all(s0, c0, 0), next = read_all(s1, c0, 1);
            while (!done) {
                for_passes<0, 2 * kImages>([&](auto ic) {
                    constexpr int i = decltype(ic)::value % kImages, round = decltype(ic)::value / kImages;
                    constexpr bool kBehindScales = i < 2;  // the scales were issued after what is waited for
                    if (done)
                        return;
#pragma unroll
                    for (int u = 0; u < SUB; u++)
                        multiply(cur.f[u], cur.s[u], std::integral_constant<int, 0>());
                    __builtin_amdgcn_sched_barrier(0);
                    arrive(std::integral_constant<int, kLoads + (kBehindScales ? kScaleLoads : 0)>(), std::false_type());
                    cur = next;
                    next = read_all(images[(i + 2) % kImages], places[i < 2 ? round : 1 - round], (i + 2) % kImages);
                    fill(images[i], n + kImages);
                    if constexpr (i == kImages - 1)
                        fill_scales(places[round], n / kImages + 2);
                    done = ++n >= all;
                });
            }
        } else {
            // The same with operands read a step ahead.
            fill_scales(c0, 0);
            fill(s0, 0);
            fill(s1, 1);
            fill(s2, 2);
            fill(s3, 3);
            fill_scales(c1, 1);
            arrive(std::integral_constant<int, 3 * kLoads + kScaleLoads>(), std::true_type());
            Operands cur = read(s0, 0);
            Scales sc = read_scales(c0, 0);
            while (!done) {
                for_passes<0, 2 * kImages>([&](auto ic) {
                    constexpr int i = decltype(ic)::value % kImages, round = decltype(ic)::value / kImages;
                    if (done)
                        return;
                    for_passes<0, kSteps>([&](auto jc) {
                        constexpr int j = decltype(jc)::value;
                        Operands next;
                        if constexpr (j + 1 < kSteps) {
                            next = read(images[i], j + 1);
                            multiply(cur, sc, jc);
                        } else {
                            // the products first: they need nothing that is still on its way
                            multiply(cur, sc, jc);
                            arrive(std::integral_constant<int, 2 * kLoads + (i < kImages - 1 ? kScaleLoads : 0)>(), std::true_type());
                            next = read(images[(i + 1) % kImages], 0);
                            sc = read_scales(places[i < 3 ? round : 1 - round], (i + 1) % kImages);
                            fill(images[i], n + kImages);
                            if constexpr (i == kImages - 1)
                                fill_scales(places[round], n / kImages + 2);
                        }
                        cur = next;
                    });
                    done = ++n >= all;
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
constexpr TileShape kTileShapes[5] = {{256, 256}, {128, 128}, {64, 64}, {64, 64}, {128, 128}};
constexpr int kDeepShape = 3, kTailShape = 4;
constexpr int kTileThreads = 256;

template <typename OT, int FORMAT>
const void *tile_fn(int shape) {
    constexpr int kWk = KTile<FORMAT>::kSteps;
    switch (shape) {
    case 0: return reinterpret_cast<const void *>(&mx_tile_kernel<OT, FORMAT, 256, 256, 2, 2>);
    case 1: return reinterpret_cast<const void *>(&mx_ring_kernel<OT, FORMAT, 128, 128, 2, 2, 1, 1>);
    case 2: return reinterpret_cast<const void *>(&mx_ring_kernel<OT, FORMAT, 64, 64, 1, 4 / kWk, kWk, 1>);
    case kTailShape: return reinterpret_cast<const void *>(&mx_tile_kernel<OT, FORMAT, 128, 128, 2, 2>);
    }
    if constexpr (FORMAT == SSU_FORMAT_MXFP8)  // kDeepShape
        return reinterpret_cast<const void *>(&mx_ring_kernel<OT, FORMAT, 64, 64, 1, 4 / kWk, kWk, 2>);
    return nullptr;
}

// The largest tile of which there are more than 128: otherwise there are at most two of the next
// smaller one for each compute unit, and they are done sooner. k 4096, in us:
//   256 and 128: 2048 x 4096 (128 of the large) 42.4 and 38.0, 2048 x 5120 (160) 39.4 and 46.8,
//     2048 x 8192 (256) 44.9 and 60.3; MXFP8 57.4 and 49.7, 55.7 and 64.9, 61.9 and 83.9
//   128 and 64: 1024 x 2048 (128) 19.7 and 17.8, 1024 x 2560 (160) 19.6 and 22.9,
//     1024 x 4096 (256) 21.0 and 27.7; MXFP8 25.2 and 24.0, 25.4 and 29.5, 26.5 and 38.8
// Of the smallest, MXFP8 takes images of two K tiles if no unit gets a second workgroup: 64 x 2048
// 14.1 instead of 15.1, but 64 x 16384 and twice the rows 25.5 instead of 20.4. MXFP4's K tiles are as
// deep by themselves (11.4 with two of them, 10.8 without).
int tile_shape(int64_t m, int64_t n, int format) {
    const auto tiles = [&](int s) { return ((m + kTileShapes[s].tm - 1) / kTileShapes[s].tm) * ((n + kTileShapes[s].tn - 1) / kTileShapes[s].tn); };
    for (int s = 0; s < 2; s++)
        if (tiles(s) > 128)
            return s;
    return format == SSU_FORMAT_MXFP8 && tiles(2) <= 256 ? kDeepShape : 2;
}

// Where the large tiles end and a second launch of smaller ones takes over: large tiles that would be
// a last round of few take a whole round's time, four times as many small ones about half of it.
// 2048 rows, k 4096, MXFP4: with 8 large tiles (of a workgroup each) left 67.8 us instead of 76.5, with 32
// 68.4 (76.7), with 96 75.4 (81.3), with 128 85.5 (85.4). They are taken from the last rows or
// columns of tiles, whichever are fewer.
struct Cut {
    int64_t m, n;  // the large tiles' rows and columns
};
constexpr int kTailMost = 96;
Cut tail_cut(int64_t m, int64_t n) {
    const int64_t mt = (m + 255) / 256, nt = (n + 255) / 256, full = mt * nt / 256 * 256;
    if (full == 0)
        return {m, n};
    const int64_t rows = full / nt, cols = full / mt;  // whole rows, or columns, of tiles in the full rounds
    const int64_t below = (mt - rows) * nt, right = (nt - cols) * mt;
    if (std::min(below, right) > kTailMost)
        return {m, n};
    return below < right ? Cut{std::min(m, rows * 256), n} : Cut{m, std::min(n, cols * 256)};
}

// Whether a smaller tile can fetch scale bytes where they are (see padded_scales).
bool scales_in_place(const void *base, int64_t stride, int64_t k) {
    return k % 512 == 0 && stride % 16 == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0;
}

template <typename F>
const void *by_out(int out_dtype, F &&f) {
    return out_dtype == SSU_F32 ? f(0.0f) : out_dtype == SSU_F16 ? f(static_cast<_Float16>(0)) : f(static_cast<__bf16>(0));
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t code_bytes(int64_t m, int64_t k, int format) { return round256(format == SSU_FORMAT_MXFP4 ? m * k / 2 : m * k); }

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
    return launch_groups(fn, blocks, kQuantThreads, args, stream);
}

int64_t mx_linear_workspace(int64_t m, int64_t n, int64_t k, int format, bool floats) {
    const int64_t codes = floats && m > kMxFuseRows ? code_bytes(m, k, format) : 0;
    if (m <= kMxRowsMax)
        return codes > 0 ? codes + m * (k / 32) : 0;
    if (tile_shape(m, n, format) == 0)
        return codes + 4 * (packed_room(m, ktiles_of(k, format)) + packed_room(n, ktiles_of(k, format)));
    return codes + (m + n) * padded_scales(k);
}

int launch_mx_linear(const MxParams &args_in, int format, int out_dtype, void *stream) {
    MxParams p = args_in;
    const bool mx4 = format == SSU_FORMAT_MXFP4;
    const bool floats = p.x != nullptr;
    if (p.m <= kMxRowsMax) {
        const bool fuse = floats && p.m <= kMxFuseRows;
        if (floats && !fuse && p.k > 0) {
            uint8_t *scales = p.workspace + code_bytes(p.m, p.k, format);
            if (int e = launch_mx_quantize_rows(p.x, p.x_dtype, p.x_s, p.m, p.k, p.workspace, scales, format, stream))
                return e;
            p.a = p.workspace;
            p.a_scale = scales;
            p.a_s = mx4 ? p.k / 2 : p.k;
            p.as_s = p.k / 32;
        }
        const void *fn = by_out(out_dtype, [&](auto o) {
            using OT = decltype(o);
            return mx4 ? stream_fn<OT, SSU_FORMAT_MXFP4>(fuse, p.x_dtype) : stream_fn<OT, SSU_FORMAT_MXFP8>(fuse, p.x_dtype);
        });
        void *args[] = {&p};
        return launch_groups(fn, (p.n + kStreamRows - 1) / kStreamRows, kStreamWaves * 64, args, stream);
    }

    const int shape = tile_shape(p.m, p.n, format);
    TileParams t = {};
    t.ktiles = static_cast<int32_t>(shape == 0 ? ktiles_of(p.k, format) : padded_scales(p.k) * 32 / ktile_depth(format));
    t.a_scales = p.a_scale;
    t.w_scales = p.w_scale;
    // one launch before the product for what has to be quantised or laid out
    PackParams q = {};
    q.m = p.m, q.n = p.n, q.k = p.k;
    q.ktiles = shape == 0 ? t.ktiles : 0;
    uint8_t *ws = p.workspace;
    int64_t a_work = 0, w_work = 0;
    if (floats) {
        q.x = p.x;
        q.x_s = p.x_s;
        q.codes = ws;
        p.a = ws;
        p.a_s = mx4 ? p.k / 2 : p.k;
        ws += code_bytes(p.m, p.k, format);
        a_work = static_cast<int64_t>(p.m) * (shape == 0 ? t.ktiles * (ktile_depth(format) / 8) : padded_scales(p.k) * 4);
    } else if (shape == 0 || !scales_in_place(p.a_scale, p.as_s, p.k)) {
        q.a_scale = p.a_scale;
        q.as_s = p.as_s;
        a_work = shape == 0 ? packed_words(p.m, t.ktiles) : p.m * padded_scales(p.k) / 4;
    }
    if (a_work > 0) {
        q.a_out = ws;
        t.a_scales = ws;
        p.as_s = padded_scales(p.k);
    }
    if (shape == 0 || !scales_in_place(p.w_scale, p.ws_s, p.k)) {
        q.w_scale = p.w_scale;
        q.ws_s = p.ws_s;
        q.w_out = ws + (shape == 0 ? 4 * packed_room(p.m, t.ktiles) : p.m * padded_scales(p.k));
        w_work = shape == 0 ? packed_words(p.n, t.ktiles) : p.n * padded_scales(p.k) / 4;
        t.w_scales = q.w_out;
        p.ws_s = padded_scales(p.k);
    }
    if (a_work + w_work > 0) {
        const auto groups = [](int64_t work) { return static_cast<int>(std::min<int64_t>((work + kQuantThreads - 1) / kQuantThreads, 32768)); };
        q.a_groups = groups(a_work);
        const void *fn = !floats                ? pack_fn<void>(format)
                         : p.x_dtype == SSU_F32 ? pack_fn<float>(format)
                         : p.x_dtype == SSU_F16 ? pack_fn<_Float16>(format)
                                                : pack_fn<__bf16>(format);
        void *args[] = {&q};
        if (int e = launch_groups(fn, q.a_groups + groups(w_work), kQuantThreads, args, stream))
            return e;
    }
    t.p = p;
    const auto launch = [&](int shape) {
        t.mtiles = (t.p.m + kTileShapes[shape].tm - 1) / kTileShapes[shape].tm;
        t.ntiles = (t.p.n + kTileShapes[shape].tn - 1) / kTileShapes[shape].tn;
        const void *fn = by_out(out_dtype, [&](auto o) {
            using OT = decltype(o);
            return mx4 ? tile_fn<OT, SSU_FORMAT_MXFP4>(shape) : tile_fn<OT, SSU_FORMAT_MXFP8>(shape);
        });
        void *args[] = {&t};
        return launch_groups(fn, static_cast<int64_t>(t.mtiles) * t.ntiles, kTileThreads, args, stream);
    };
    if (shape != 0)
        return launch(shape);
    const Cut cut = tail_cut(p.m, p.n);
    t.p.m = static_cast<int32_t>(cut.m);
    t.p.n = static_cast<int32_t>(cut.n);
    if (int e = launch(0))
        return e;
    if (cut.m == p.m && cut.n == p.n)
        return 0;
    const int64_t out_bytes = out_dtype == SSU_F32 ? 4 : 2;
    if (cut.m < p.m) {
        t.p.m = static_cast<int32_t>(p.m - cut.m);
        t.p.a += cut.m * p.a_s;
        t.a_scales += 4 * packed_words(cut.m, t.ktiles);
        t.p.out = static_cast<char *>(t.p.out) + cut.m * p.out_s * out_bytes;
    } else {
        t.p.n = static_cast<int32_t>(p.n - cut.n);
        t.p.w += cut.n * p.w_s;
        t.w_scales += 4 * packed_words(cut.n, t.ktiles);
        t.p.out = static_cast<char *>(t.p.out) + cut.n * out_bytes;
        if (p.bias)
            t.p.bias = static_cast<const char *>(p.bias) + cut.n * (p.bias_f32 ? 4 : out_bytes);
    }
    return launch(kTailShape);
}

}  // namespace ssu
