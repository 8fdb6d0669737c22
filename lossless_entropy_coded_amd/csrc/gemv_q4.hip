// gemv_q4.hip -- matrix-vector products with 4-bit weights and group scales,
// the consumer of int4 code planes:
//
//   y[t][r] = sum_c scale[r][c / group] (code[r][c] - zero[r][c / group]) x[t][c]
//
// for 1..16 vectors x[t] (one token, or the few that are verified at once).
// Codes are two per byte, the first in the low nibble; zero points are 8 where
// none are given.
//
// A product of this kind reads every weight once and is bound by memory, if the
// vector units keep up: at 8 TB/s a CU has 2.4 operations per weight, and
// converting and multiplying weights one at a time takes that for one vector
// and more for each further one.  So the products are the matrix cores':
//   - v_mfma_f32_16x16x32_f16, its 16 rows the vectors (those not there are
//     zero), its 16 columns weight rows, 32 columns of W at a time;
//   - code less zero point is made exactly in f16, two at a time: a nibble put
//     into the mantissa of 1024 is 1024 + code (four bits higher: 1024 + 16
//     code), and one packed addition of -(1024 + zero) (or one packed fma, by
//     1 / 16, of -(64 + zero)) leaves the difference: 9 operations per 8
//     weights whatever the zero point and the number of vectors;
//   - x is scaled by a power of two, so that the largest value of a vector's
//     slab of 128 to 512 columns is just below 2^16, and put into f16.  That
//     is exact for values down to 2^-32 of the largest (a bf16 value has 8
//     significant bits), and off by less than 2^-39 of it below; an infinity
//     or NaN stays one;
//   - the products are exact in fp32 and sums are held in fp32: a group's sum
//     times its scale is added to the slab's, the slab's to the row's.  The
//     slab's power of two goes back in before the scale where it is below one,
//     after it where it is above: so nothing on the way leaves fp32's range that
//     the plain products would not (a sum is up to 2^31 before it, scales are
//     any finite bf16).  Neither loses bits: sums below 2^-126 are multiples of
//     x's smallest steps, which fp32 holds.
// (Subtracting zero * sum(x) from sum(code x) instead would lose small products
// next to a large x that its zero point cancels.  bf16 in place of f16, code
// by code through v_cvt_off_f32_i4, needs no scaling of x but 1.75 operations
// per weight, 2.4 with zero points: 12.2 us at 14336 x 4096, one vector, where
// this takes 9.8.)
//
// A wave takes 16 kTiles rows and a part of the columns, 128 columns per step.
// Lane 4 r + q loads the 16 bytes of row r's q-th chunk of 32 columns, so that
// four neighbouring lanes read 64 neighbouring bytes: memory instructions take
// as long as their quads of lanes touch cache lines.  Through LDS the chunk
// goes to lane 16 q + r, as the matrix operand wants it; four rows of lanes
// exchange dwords (2 + 2 lane swaps) so that each of the four products of a
// step has 32 neighbouring columns; and x comes through the wave's own LDS too.
// The waves of a workgroup share the rows and split the columns, and add their
// sums in order at the end: everything is summed in a fixed order.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "buffers.h"

namespace wc {
namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kStepCols = 128;
constexpr uint32_t kMaxWaves = 8;

struct Q4Params {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    const uint16_t* x;
    float* y;
    uint32_t rows, cols, group, groups, vecs;
    uint32_t group_magic;      // chunk / (group / 32) = mulhi(chunk, group_magic) + (chunk & group_one)
    uint32_t group_one;
    uint32_t slabs_per_wave;
};

// A slab is what a wave has on its way at a time: kSlab steps.  LDS of one wave:
// x of a slab in f16, [vector][column], and 2^(E - 15) of each vector, 2^E the
// largest power of two in its slab.
template <int kVecs>
struct Q4Shape {
    static constexpr uint32_t kSlab = kVecs == 1 ? 4 : kVecs == 16 ? 1 : 2;
    static constexpr uint32_t kRowBytes = kSlab * kStepCols * 2;   // of one vector
    static constexpr uint32_t kRounds = kVecs * kSlab / 4;         // 64 lanes of 8 columns
    static constexpr uint32_t kXBytes = kVecs * kRowBytes;
    static constexpr uint32_t kWaveBytes = kXBytes + 64;
    static constexpr uint32_t kSwapBytes = 1024;                   // per tile, of each wave
    static constexpr uint32_t kNoneBytes = kSlab * 256;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, kBufferWord);
}

// Constants in registers: an operation takes no second literal, and with these
// "and" and "or" are one.
struct Consts {
    uint32_t low = 0x000F000Fu, high = 0x00F000F0u, magic = 0x64006400u;
    __device__ __forceinline__ Consts() { asm("" : "+s"(low), "+s"(high), "+v"(magic)); }
};

// code - zero point in f16 for the 8 codes of a dword, in the order 0 4 1 5 2 6 3 7; by1: -(1024 + zero point), by16:
// -(64 + zero point), both twice.
__device__ __forceinline__ f16x8 weights(uint32_t codes, f16x2 by1, f16x2 by16, const Consts& k) {
    const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    f16x2 w[4];
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i, codes >>= 8) {
        w[2 * i] = __builtin_bit_cast(f16x2, (codes & k.low) | k.magic) + by1;
        w[2 * i + 1] = __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (codes & k.high) | k.magic), sixteenth, by16);
    }
    return __builtin_bit_cast(f16x8, u32x4{__builtin_bit_cast(uint32_t, w[0]), __builtin_bit_cast(uint32_t, w[1]),
                                           __builtin_bit_cast(uint32_t, w[2]), __builtin_bit_cast(uint32_t, w[3])});
}

// The largest value of the lanes in 16 kRows lanes.
template <int kRows>
__device__ __forceinline__ uint32_t largest(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));    // lane ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));    // lane ^ 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));   // half row mirrored
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));   // row mirrored
    if (kRows >= 2) {
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));
        v = max(a.x, a.y);
    }
    if (kRows >= 4) {
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
        v = max(a.x, a.y);
    }
    return v;
}

// Transposes four dwords of four rows of 16 lanes: out[j] in row q is in[q] of row j.
__device__ __forceinline__ u32x4 transpose_rows(const u32x4& in) {
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(in[0], in[2], false, false));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(in[1], in[3], false, false));
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a.x, b.x, false, false));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a.y, b.y, false, false));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// out[j]: row j's value, in all four rows of 16 lanes.
__device__ __forceinline__ u32x4 spread_rows(uint32_t v) {
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v, v, false, false));
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a.x, a.x, false, false));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a.y, a.y, false, false));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
}

// What a wave has in registers for one slab: its codes, scale bits and zero
// points, and x.  A row's scales, of the slab's blocks of kBlock chunks, are
// loaded four at a time, one by each row of lanes: loads of two bytes by 64
// lanes cost as much as loads of sixteen (one per step: 12.2 us at 14336 x
// 4096, one vector; without any: 7.4).
// kFour: a row's four scales of a step stand side by side and are loaded as one,
// a step's by each row of lanes.
template <int kVecs, int kTiles, int kBlock, bool kFour>
struct Slab {
    using S = Q4Shape<kVecs>;
    static constexpr uint32_t kBlocks = S::kSlab * 4 / kBlock, kScales = (kBlocks + 3) / 4;
    u32x4 w[S::kSlab][kTiles];
    uint32_t scale[kFour ? 2 : kScales][kTiles];
    uint32_t zero[kFour ? 1 : kScales][kTiles];
    u32x4 x[S::kRounds];
};

// kVecs: vectors, rounded up.  kBlock: chunks of 32 columns (1, 2 or 4) that
// always share a group.  kWhole: columns are a multiple of 32, so that a lane's
// chunk is one 16-byte load; kZeros: zero points are given (they may be, if
// not kWhole).
template <int kVecs, int kTiles, int kBlock, bool kFour, bool kWhole, bool kZeros>
__global__ __launch_bounds__(64 * kMaxWaves) void gemv_q4_kernel(Q4Params p) {
    using S = Q4Shape<kVecs>;
    constexpr bool kGiven = kZeros || !kWhole;
    using Loads = Slab<kVecs, kTiles, kBlock, kFour>;
    extern __shared__ __align__(16) uint8_t lds[];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t waves = blockDim.x >> 6;
    uint8_t* const xs = lds + wave * (S::kWaveBytes + kTiles * S::kSwapBytes);
    uint8_t* const swap = xs + S::kWaveBytes;
    float* const units = reinterpret_cast<float*>(xs + S::kXBytes);
    uint8_t* const none = lds + waves * (S::kWaveBytes + kTiles * S::kSwapBytes);   // zeros, for vectors that are not there
    for (uint32_t i = threadIdx.x; i < S::kNoneBytes / 4; i += blockDim.x) reinterpret_cast<uint32_t*>(none)[i] = 0;
    if (lane < 16) units[lane] = 0.0f;
    __syncthreads();

    const uint32_t r = lane & 15u, q = lane >> 4;   // weight row of a tile (or vector, holding x); chunk of a step
    const uint32_t lr = lane >> 2, lq = lane & 3u;  // the same, loading
    const uint32_t row0 = blockIdx.x * 16 * kTiles, rows = min(p.rows - row0, 16u * kTiles);
    const uint32_t row_bytes = p.cols / 2;
    const auto codes_buf = buffer(p.codes + (uint64_t)row0 * row_bytes, (uint64_t)rows * row_bytes);
    const auto scale_buf = buffer(p.scales + (uint64_t)row0 * p.groups, (uint64_t)rows * p.groups * 2);
    const auto zero_buf = buffer(p.zeros + (uint64_t)row0 * p.groups, p.zeros ? (uint64_t)rows * p.groups : 0);
    const uint32_t no_zeros = p.zeros ? 0 : 8;
    const auto x_buf = buffer(p.x, (uint64_t)p.vecs * p.cols * 2);
    uint32_t code_at[kTiles], group_at[kTiles];   // of the lane's rows; those past the last repeat it
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        const uint32_t row = min(i * 16 + lr, rows - 1);
        code_at[i] = row * row_bytes + lq * 16;
        group_at[i] = row * p.groups;
    }

    // Where the lane reads its vector's x.  64-byte pieces of a step stand at piece ^ (vector & 3), so that four
    // vectors' lie in different banks.
    const bool there = r < (uint32_t)kVecs;
    const uint8_t* x_at[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
        x_at[j] = there ? xs + r * S::kRowBytes + q * 16 + ((j ^ (r & 3u)) * 64) : none;

    // from lane 4 r + q to lane 16 q + r: 16-byte pieces of a row at piece ^ (row / 4), in different banks
    uint8_t* const swap_to = swap + lr * 64 + ((lq ^ (lr >> 2)) * 16);
    const uint8_t* const swap_from = swap + r * 64 + ((q ^ (r >> 2)) * 16);
    const int word_from = (int)(r * 4 + q) * 4;

    uint32_t x_from[S::kRounds];
#pragma unroll
    for (uint32_t round = 0; round < S::kRounds; ++round) {
        const uint32_t job = round * 4 + q, v = job / S::kSlab;
        x_from[round] = v < p.vecs ? (v * p.cols + job % S::kSlab * kStepCols + r * 8) * 2 : kNoChunk;
    }

    // Start the loads of a slab.  The uniform part of an offset stays within the buffer: past its end (in the last
    // slab, or the one after it) the range check of a lane's part, which subtracts it, could wrap.
    const auto load = [&](uint32_t slab) {
        Loads l;
        const uint32_t c0 = slab * S::kSlab * kStepCols;
#pragma unroll
        for (uint32_t round = 0; round < S::kRounds; ++round) {
            const uint32_t c = c0 + (round * 4 + q) % S::kSlab * kStepCols + r * 8;
            l.x[round] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                x_buf, c < p.cols ? x_from[round] : kNoChunk, min(c0, p.cols) * 2, 0));
        }
#pragma unroll
        for (uint32_t st = 0; st < S::kSlab; ++st) {
            const uint32_t cs = c0 + st * kStepCols, c = cs + lq * 32, uniform = min(cs, p.cols) / 2;
            const bool inside = c < p.cols;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                if (kWhole) {
                    l.w[st][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                        codes_buf, inside ? code_at[i] : kNoChunk, uniform, 0));
                } else {
#pragma unroll
                    for (uint32_t d = 0; d < 4; ++d)
                        l.w[st][i][d] = __builtin_amdgcn_raw_buffer_load_b32(
                            codes_buf, c + d * 8 < p.cols ? code_at[i] + d * 4 : kNoChunk, uniform, 0);
                }
            }
        }
        if constexpr (kFour) {
            const uint32_t first = min(slab * S::kSlab + min(lq, S::kSlab - 1), p.cols / kStepCols - 1) * 4;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const u32x2 s4 = __builtin_bit_cast(
                    u32x2, __builtin_amdgcn_raw_buffer_load_b64(scale_buf, (group_at[i] + first) * 2, 0, 0));
                l.scale[0][i] = s4.x, l.scale[1][i] = s4.y;
                l.zero[0][i] = kGiven ? __builtin_amdgcn_raw_buffer_load_b32(zero_buf, group_at[i] + first, 0, 0) : 0;
            }
        } else
#pragma unroll
        for (uint32_t k = 0; k < Loads::kScales; ++k) {
            const uint32_t block = k * 4 + min(lq, Loads::kBlocks - 1);
            const uint32_t chunk = min(c0 + block * kBlock * 32, p.cols - 1) / 32;
            const uint32_t g = __umulhi(chunk, p.group_magic) + (chunk & p.group_one);
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                l.scale[k][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(scale_buf, (group_at[i] + g) * 2, 0, 0);
                l.zero[k][i] =   // the buffer is empty where none are given
                    kGiven ? (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(zero_buf, group_at[i] + g, 0, 0) + no_zeros : 8u;
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // started before what is multiplied next
        return l;
    };

    const Consts consts;
    f32x4 acc[kTiles];   // of weight row r and vectors 4 q ..  4 q + 3
#pragma unroll
    for (int i = 0; i < kTiles; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const auto exchanged = [&](uint32_t v) { return (uint32_t)__builtin_amdgcn_ds_bpermute(word_from, (int)v); };
    const auto process = [&](const Loads& l) {
        // x to f16, 8 columns per lane
#pragma unroll
        for (uint32_t round = 0; round < S::kRounds; ++round) {
            const uint32_t job = round * 4 + q, v = job / S::kSlab, st = job % S::kSlab;
            const u32x4 xw = l.x[round];
            u16x2 m = __builtin_bit_cast(u16x2, xw[0] & 0x7FFF7FFFu);
#pragma unroll
            for (uint32_t i = 1; i < 4; ++i)
                m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, xw[i] & 0x7FFF7FFFu));
            const int e = (int)(largest<S::kSlab>(max((uint32_t)m.x, (uint32_t)m.y)) >> 7);   // E + 127
            u32x4 to;
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {   // columns i and i + 4
                const float lo = __uint_as_float(i & 1 ? xw[i / 2] & 0xFFFF0000u : xw[i / 2] << 16);
                const float hi = __uint_as_float(i & 1 ? xw[i / 2 + 2] & 0xFFFF0000u : xw[i / 2 + 2] << 16);
                to[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(__builtin_ldexpf(lo, 142 - e),
                                                                               __builtin_ldexpf(hi, 142 - e)));
            }
            *reinterpret_cast<u32x4*>(xs + v * S::kRowBytes + st * 256 + ((r * 16) ^ ((v & 3u) * 64))) = to;
            if (st == 0 && r == 0) units[v] = __builtin_ldexpf(1.0f, e - 142);
        }
        // the wave's lanes exchange x through its own LDS, which it accesses in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();

        u32x4 words[Loads::kScales][kTiles];   // scale bits << 16 | zero point of four blocks, in every row of lanes
        if constexpr (kFour) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                u32x4 own;   // of the row of lanes' step
#pragma unroll
                for (uint32_t b = 0; b < 4; ++b) {
                    const uint32_t two = l.scale[b / 2][i];
                    own[b] = exchanged((b & 1 ? two & 0xFFFF0000u : two << 16) |
                                       (kGiven ? (l.zero[0][i] >> (8 * b)) & 0xFFu : 0));
                }
                own = transpose_rows(own);
#pragma unroll
                for (uint32_t k = 0; k < Loads::kScales; ++k) words[k][i] = spread_rows(own[k]);
            }
        } else {
#pragma unroll
            for (uint32_t k = 0; k < Loads::kScales; ++k)
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
                    words[k][i] =
                        spread_rows(exchanged(kGiven ? l.scale[k][i] << 16 | l.zero[k][i] : l.scale[k][i] << 16));
        }
        const u32x4 unit = *reinterpret_cast<const u32x4*>(units + q * 4);   // of vectors 4 q .., the bits
        f32x4 below, above;   // the part of it below one, and that above
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            below[e] = __uint_as_float(min(unit[e], 0x3F800000u)), above[e] = __uint_as_float(max(unit[e], 0x3F800000u));
        f32x4 sum[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) sum[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (uint32_t st = 0; st < S::kSlab; ++st) {
            f16x8 x[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const f16x8*>(x_at[j] + st * 256);
#pragma unroll
            for (int i = 0; i < kTiles; ++i) *reinterpret_cast<u32x4*>(swap_to + i * S::kSwapBytes) = l.w[st][i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            u32x4 chunk[kTiles];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) chunk[i] = *reinterpret_cast<const u32x4*>(swap_from + i * S::kSwapBytes);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const u32x4 w = transpose_rows(chunk[i]);
#pragma unroll
                for (uint32_t b = 0; b < 4 / kBlock; ++b) {
                    const uint32_t block = st * (4 / kBlock) + b, word = words[block / 4][i][block % 4];
                    const uint32_t z = kGiven ? word & 0xFFu : 8u;
                    const float scale = __uint_as_float(word & 0xFFFF0000u);
                    const f16x2 by1 = __builtin_bit_cast(f16x2, z * 0x00010001u + 0xE400E400u);
                    const f16x2 by16 = by1 + f16x2{(_Float16)960.0f, (_Float16)960.0f};
                    f32x4 D = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (uint32_t j = b * kBlock; j < (b + 1) * kBlock; ++j)
                        D = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[j], weights(w[j], by1, by16, consts), D, 0, 0, 0);
#pragma unroll
                    for (uint32_t e = 0; e < 4; ++e) sum[i][e] = __builtin_fmaf(D[e] * below[e], scale, sum[i][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(sum[i][e], above[e], acc[i][e]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };

    // The next slab is on its way while one is multiplied.  Workgroups begin at different slabs of their part: rows
    // lie a power of two apart more often than not, so that the same columns of all rows share a few memory
    // channels, which all workgroups would use at the same time.
    const uint32_t steps = (p.cols + kStepCols - 1) / kStepCols, slabs = (steps + S::kSlab - 1) / S::kSlab;
    const uint32_t begin = wave * p.slabs_per_wave, end = min(begin + p.slabs_per_wave, slabs);
    const uint32_t count = end > begin ? end - begin : 0;
    uint32_t at = count ? blockIdx.x % count : 0;
    const auto following = [&](uint32_t i) { return i + 1 < count ? i + 1 : 0; };
    Loads one = load(begin + at);
    for (uint32_t i = 0; i < count; i += 2) {
        const uint32_t at1 = following(at), at2 = following(at1);
        const Loads two = load(i + 1 < count ? begin + at1 : slabs);   // past the last one: zeros
        process(one);
        if (i + 1 >= count) break;
        one = load(i + 2 < count ? begin + at2 : slabs);
        process(two);
        at = at2;
    }

    // the waves in order
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(lds);   // [wave][kVecs][16 kTiles]
    constexpr uint32_t kOut = kVecs * 16 * kTiles;
    static_assert(kOut * 4 <= S::kWaveBytes + kTiles * S::kSwapBytes, "the sums fit where x was");
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            if (q * 4 + e < kVecs) sums[wave * kOut + (q * 4 + e) * 16 * kTiles + i * 16 + r] = acc[i][e];
    __syncthreads();
    for (uint32_t o = threadIdx.x; o < kOut; o += blockDim.x) {
        const uint32_t v = o / (16 * kTiles), row = row0 + o % (16 * kTiles);
        if (v >= p.vecs || row >= p.rows) continue;
        float sum = sums[o];
        for (uint32_t k = 1; k < waves; ++k) sum += sums[k * kOut + o];
        p.y[(uint64_t)v * p.rows + row] = sum;
    }
}

template <int kVecs, int kTiles>
void launch(Q4Params& p, uint32_t waves, hipStream_t s) {
    using S = Q4Shape<kVecs>;
    const uint32_t steps = (p.cols + kStepCols - 1) / kStepCols, slabs = (steps + S::kSlab - 1) / S::kSlab;
    waves = waves < slabs ? waves : slabs;
    p.slabs_per_wave = (slabs + waves - 1) / waves;
    waves = (slabs + p.slabs_per_wave - 1) / p.slabs_per_wave;
    const dim3 grid((p.rows + 16 * kTiles - 1) / (16 * kTiles)), block(64 * waves);
    const uint32_t bytes = waves * (S::kWaveBytes + kTiles * S::kSwapBytes) + S::kNoneBytes;
    const auto go = [&](auto* kernel) { hipLaunchKernelGGL(kernel, grid, block, bytes, s, p); };
    if (p.cols % 32 != 0) return go(gemv_q4_kernel<kVecs, kTiles, 1, false, false, true>);
    const bool zeros = p.zeros;
    const bool four = p.group == 32 && p.cols % kStepCols == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 7u) == 0 &&
                      (reinterpret_cast<uintptr_t>(p.zeros) & 3u) == 0;
    if (p.group % 128 == 0 || p.group >= p.cols)
        zeros ? go(gemv_q4_kernel<kVecs, kTiles, 4, false, true, true>)
              : go(gemv_q4_kernel<kVecs, kTiles, 4, false, true, false>);
    else if (p.group % 64 == 0)
        zeros ? go(gemv_q4_kernel<kVecs, kTiles, 2, false, true, true>)
              : go(gemv_q4_kernel<kVecs, kTiles, 2, false, true, false>);
    else if (four)
        zeros ? go(gemv_q4_kernel<kVecs, kTiles, 1, true, true, true>)
              : go(gemv_q4_kernel<kVecs, kTiles, 1, true, true, false>);
    else
        zeros ? go(gemv_q4_kernel<kVecs, kTiles, 1, false, true, true>)
              : go(gemv_q4_kernel<kVecs, kTiles, 1, false, true, false>);
}

// Rows and waves per workgroup.  From 8192 rows on there are workgroups enough
// of 16 rows and 4 waves, or of 32 rows, which share the work on x, where
// vectors make that count, and then of 8 waves from 5 vectors on; below, 16 rows
// and 8 waves, which split the columns further.  Measured on matrices that rotate
// past the caches, groups of 128 (32 for 2088 columns), us:
//                                        16 rows        32 rows
//                                   4 waves 8 waves 4 waves 8 waves
//   14336 x 4096, one vector           10.9    12.3    11.8    13.0
//   10240 x 4096, one vector            8.8     9.7    11.3    12.3
//    8192 x 4096, one vector            7.3     7.5     8.1     7.9
//    6144 x 4096, one vector            6.9     7.0     7.4     7.3
//    4096 x 14336, one vector          11.3    10.0    15.4    16.1
//   14336 x 4096, 4 vectors            12.1    12.9    11.6    11.8
//    8192 x 4096, 4 vectors             8.1     8.0     8.2     8.1
//    6144 x 4096, 4 vectors             7.9     7.9     8.0     7.8
//    4096 x 14336, 4 vectors           16.0    12.1    19.1    16.3
//   14336 x 4096, 16 vectors           19.7    20.1    16.1    15.7
//    8192 x 28672, 8 vectors           44.6    43.6    41.7    38.1
//    8192 x 4096, 8 vectors             9.7    10.0     9.3     9.2
//    6144 x 4096, 8 vectors             9.6     9.8     9.1     8.8
//    4096 x 4096, 8 vectors             7.8     6.8     8.9     8.5
//    1003 x 2088, 4 vectors             6.4     5.5     8.6     7.4
// (At 6144 rows 32 already gain a tenth for 8 vectors and more.)
template <int kVecs>
void launch_rows(Q4Params& p, hipStream_t s) {
    if (p.rows < 8192) return launch<kVecs, 1>(p, 8, s);
    if constexpr (kVecs >= 4)
        launch<kVecs, 2>(p, kVecs >= 8 ? 8 : 4, s);
    else
        launch<kVecs, 1>(p, 4, s);
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wc_q4_check(const wc_q4_matrix* W) {
    if (!W || W->cols == 0 || W->cols % 8 != 0 || W->cols > WC_MAX_DIM || W->group == 0 || W->group % 32 != 0 ||
        W->rows > WC_MAX_VOCAB)
        return WC_ERR_INVALID_ARG;
    if (W->rows == 0) return WC_OK;
    if (!W->codes || (reinterpret_cast<uintptr_t>(W->codes) & 15u) || !W->scales ||
        (reinterpret_cast<uintptr_t>(W->scales) & 1u))
        return WC_ERR_INVALID_ARG;
    return WC_OK;
}

extern "C" int wc_gemv_q4_async(const wc_q4_matrix* W, const uint16_t* x, uint32_t n_vecs, float* y, void* stream) {
    const int st = wc_q4_check(W);
    if (st != WC_OK) return st;
    if (n_vecs > WC_GEMV_Q4_MAX_VECS) return WC_ERR_INVALID_ARG;
    if (W->rows == 0 || n_vecs == 0) return WC_OK;
    if (!x || !y || (reinterpret_cast<uintptr_t>(x) & 15u) || (reinterpret_cast<uintptr_t>(y) & 3u))
        return WC_ERR_INVALID_ARG;
    Q4Params p{};
    p.codes = W->codes, p.scales = W->scales, p.zeros = W->zeros, p.x = x, p.y = y;
    p.rows = W->rows, p.cols = W->cols, p.group = W->group, p.vecs = n_vecs;
    p.groups = W->group < W->cols ? (W->cols + W->group - 1) / W->group : 1;
    // ceil(2^32 / m), m chunks per group: exact for fewer than 2^16 chunks of m < 2^16 (there are 2^11 at most)
    const uint32_t m = W->group < W->cols ? W->group / 32 : 1u << 15;
    p.group_magic = m == 1 ? 0 : (uint32_t)((0x100000000ull + m - 1) / m);
    p.group_one = m == 1 ? ~0u : 0;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (n_vecs == 1) launch_rows<1>(p, s);
    else if (n_vecs == 2) launch_rows<2>(p, s);
    else if (n_vecs <= 4) launch_rows<4>(p, s);
    else if (n_vecs <= 8) launch_rows<8>(p, s);
    else launch_rows<16>(p, s);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
