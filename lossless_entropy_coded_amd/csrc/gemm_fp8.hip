// gemm_fp8.hip -- products with matrices of e4m3 codes that have a scale per
// block of 128 x 128, of activations that have one per token and 128 columns:
//
//   y[t][r] = sum_b xs[t][b] ws[r / 128][b] sum_{c in block b} xc[t][c] wc[r][c].
//
// The inner sum is that of matrix instructions of 16 rows and 16 tokens, from
// zero, which is then added to the fp32 result times the product of the scales: a
// lane of its result has one token and 4 rows of one block, so that a stage of 128
// columns takes one product of scales per token and lane.
//
// Which matrix instructions: those of 8-bit operands sum 8 products at a time, and
// drop what lies 2^14 times below the largest of the eight (measured: beside 448 *
// 448, which is 1.5 * 2^17, a product of 2^3 counts and one of 2^2 does not; sums
// of eights are fp32).  On normal values that leaves the sums 1.3e-5 off, on ones
// with outliers 3e-5.  Results in bf16, themselves rounded by up to 2^-8, take that
// for twice the rate; fp32 results do not: their codes are made bf16 first, which
// is exact, and multiplied by instructions whose sums are fp32.  So are few tokens'
// codes, whose products are bound by reading the matrix either way.
//
// Of 16 x 16 x 128 with 4 multiply-adds each, on registers alone, the card sustains 3990 TFLOP/s at its power limit (without
// them 4460); of 32 x 32 x 64 with theirs 3580.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "e4m3.h"
#include "gemm_fp8_plan.h"
#include "lds_copy.h"
#include "tiles.h"

namespace wc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef const __attribute__((address_space(4))) float constant_float;   // no kernel here writes it: scalar loads

struct GemmParams {
    const uint8_t* w;
    const float* ws;
    const uint8_t* x;
    const float* xs;
    void* y;
    float* part;              // splits > 1: [split][token][row]
    uint32_t rows, cols, tokens, blocks;
    uint32_t split_blocks;    // blocks of columns per split
    uint32_t splits, out_kind;
};

// A stage in LDS: R rows of 128 codes, 8 chunks of 16 bytes, chunk c at place c ^ (row / 2 & 7), so that the 16 rows
// of one chunk that a pass of a 16-byte read touches lie in different banks.
template <uint32_t R, uint32_t kThreads>
struct Loader {
    static constexpr uint32_t kLoads = R * 8 / kThreads, kRows = kThreads / 8;   // rounds, rows of each
    static_assert(R * 8 % kThreads == 0 && kRows % 16 == 0, "whole rounds, all of the same place in their rows");
    u32x4 rsrc;
    uint32_t cols, column, at;
    __device__ __forceinline__ Loader(const uint8_t* p, uint32_t cols_, uint32_t row0, uint32_t rows) : cols(cols_) {
        const uint32_t thread = threadIdx.x % kThreads;
        rsrc = buffer_words(p + (uint64_t)row0 * cols, (rows - row0 < R ? rows - row0 : R) * cols);   // row0 < rows
        const uint32_t row = thread / 8;
        column = ((thread & 7u) ^ (row / 2 & 7u)) * 16;
        at = row * cols + column;
    }
    // Start copying the stage of columns c0 .. c0 + 127 (zeros past the last): every kEvery-th round from kFirst on.  The
    // uniform part of an offset stays within the buffer: past its end the range check of a lane's part, which subtracts
    // it, would wrap.
    template <uint32_t kFirst = 0, uint32_t kEvery = 1, bool kOnce = false>
    __device__ __forceinline__ void start(uint8_t* lds, uint32_t c0) const {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % (kThreads / 64);
        const uint32_t from = c0 + column < cols ? at : kNoChunk;
#pragma unroll
        for (uint32_t i = kFirst; i < kLoads; i += kEvery) {
            const uint32_t to = lds_address(lds) + (i * kThreads + wave * 64u) * 16u;
            const uint32_t uniform = min(i * kRows * cols + c0, rsrc[2]);
            kOnce ? copy_once_to_lds(to, rsrc, from, uniform) : copy_to_lds(to, rsrc, from, uniform);
        }
    }
};

// Rows x .. x + 15 of a stage: lane l has row x + l % 16, chunks l / 16 and l / 16 + 4.  (Which columns a lane has is
// of no account as long as both operands agree.)  Where they stand; 16 rows further on, 2048 bytes further on.
struct Places {
    uint32_t lo, hi;
    __device__ __forceinline__ explicit Places(uint32_t x) {
        const uint32_t lane = threadIdx.x & 63u, row = x + (lane & 15u), at = row / 2 & 7u;
        lo = row * 128 + ((lane >> 4) ^ at) * 16;
        hi = row * 128 + ((lane >> 4 | 4u) ^ at) * 16;
    }
};
__device__ __forceinline__ i32x8 joined(const uint8_t* lo, const uint8_t* hi) {
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(*reinterpret_cast<const u32x4*>(lo),
                                                             *reinterpret_cast<const u32x4*>(hi), 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ i32x8 fragment(const uint8_t* stage, uint32_t x) {
    const Places at(x);
    return joined(stage + at.lo, stage + at.hi);
}

// Eight codes in bf16, exactly.
__device__ __forceinline__ bf16x8 widened(int lo, int hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A fragment as the products take it: as it is, or in bf16.
template <bool kExact>
struct Operand {
    i32x8 codes;
    __device__ __forceinline__ explicit Operand(const i32x8& f) : codes(f) {}
    __device__ __forceinline__ static f32x4 product(const Operand& a, const Operand& b) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.codes, b.codes, (f32x4)(0.0f), 0, 0, 0, 0, 0, 0);
    }
};
template <>
struct Operand<true> {
    bf16x8 part[4];
    __device__ __forceinline__ explicit Operand(const i32x8& f) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) part[k] = widened(f[2 * k], f[2 * k + 1]);
    }
    __device__ __forceinline__ static f32x4 product(const Operand& a, const Operand& b) {
        f32x4 d = (f32x4)(0.0f);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.part[k], b.part[k], d, 0, 0, 0);
        return d;
    }
};

// A workgroup's tile: kBm rows of the matrix by kBn tokens, over kWavesM x kWavesN waves; kGroups such groups of waves
// take blocks of columns in turn.
template <uint32_t kBm_, uint32_t kBn_, uint32_t kWavesM_, uint32_t kWavesN_, uint32_t kStages_, uint32_t kGroups_>
struct Tile {
    static constexpr uint32_t kBm = kBm_, kBn = kBn_, kWavesM = kWavesM_, kWavesN = kWavesN_, kStages = kStages_;
    static constexpr uint32_t kGroups = kGroups_, kWaves = kWavesM * kWavesN, kGroupThreads = 64 * kWaves;
    static constexpr uint32_t kThreads = kGroupThreads * kGroups;
    static constexpr uint32_t kWaveM = kBm / kWavesM, kWaveN = kBn / kWavesN;
    static constexpr uint32_t kMi = kWaveM / 16, kNi = kWaveN / 16;
    // of a stage, one group's codes, and behind all codes one group's scales: 64 tokens' per wave
    static constexpr uint32_t kCodeBytes = (kBm + kBn) * 128, kScaleBytes = kGroupThreads * 4;
    static constexpr uint32_t kScalesAt = kStages * kGroups * kCodeBytes;
    static constexpr uint32_t kLdsBytes = kScalesAt + kStages * kGroups * kScaleBytes;
    static_assert(kWaveN <= 64 && kBlockCols % kWaveM == 0 && kLdsBytes <= 160 * 1024, "shape");
};

// Four neighbouring results of a token, those past the last row left out.
__device__ __forceinline__ void store4(void* y, uint32_t kind, uint64_t at, uint32_t left, const f32x4& v) {
    if (kind == WC_OUT_F32) {
        float* const out = static_cast<float*>(y) + at;
        if (left >= 4 && (at & 3u) == 0) {
            *reinterpret_cast<f32x4*>(out) = v;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (e < left) out[e] = v[e];
        }
    } else {
        uint16_t* const out = static_cast<uint16_t*>(y) + at;
        const u32x2 w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        if (left >= 4 && (at & 3u) == 0) {
            *reinterpret_cast<u32x2*>(out) = w;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                if (e < left) out[e] = (uint16_t)(w[e / 2] >> (e % 2 * 16));
        }
    }
}

// A tile's results: put together in LDS, which is free (4 neighbours of a token per lane, 16-byte chunks at chunk ^
// token, so that the 16 tokens that a wave writes at a time lie in different banks), then written as whole rows, 16 bytes
// per lane, or where rows do not begin on 16 bytes, 4.  From the registers, 32 bytes of a token at a time, that took 10 %
// of the time at 8192 tokens x 28672 x 8192; of 3852 tokens x 18307 x 1824 it took 221 us, and so 181 (18304 rows: 161).
template <class T, uint32_t kKind>
__device__ __forceinline__ void store_tile(uint8_t* lds, void* y, const GemmParams& p, uint32_t m0, uint32_t n0,
                                           const f32x4 (&acc)[T::kMi][T::kNi]) {
    constexpr uint32_t kSize = kKind == WC_OUT_F32 ? 4 : 2, kRow = T::kBm * kSize, kChunks = kRow / 16;
    constexpr uint32_t kTurn = kChunks < 16 ? kChunks - 1 : 15;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t wm = wave % T::kWavesM * T::kWaveM, wn = wave / T::kWavesM * T::kWaveN;
    const bool holds = wave < T::kWaves;   // the first group
    // as many tokens at a time as LDS holds
    constexpr uint32_t kPass = T::kBn * kRow <= T::kScalesAt ? T::kBn : T::kBn / 2;
    static_assert(kPass * kRow <= T::kScalesAt && kPass % T::kWaveN == 0 && kPass <= T::kThreads, "a wave's tokens go together");
    static_assert((kChunks & (kChunks - 1)) == 0, "chunks are permuted");
    for (uint32_t from = 0; from < T::kBn; from += kPass) {
        if (from) __syncthreads();
        if (holds && wn >= from && wn < from + kPass) {
#pragma unroll
            for (uint32_t j = 0; j < T::kNi; ++j)
#pragma unroll
                for (uint32_t i = 0; i < T::kMi; ++i) {
                    const uint32_t n = wn - from + j * 16 + (lane & 15u), m = wm + i * 16 + (lane >> 4) * 4;
                    uint8_t* const to = lds + n * kRow + (((m * kSize / 16) ^ (n & kTurn)) * 16) + m * kSize % 16;
                    if (kSize == 4) *reinterpret_cast<f32x4*>(to) = acc[i][j];
                    else
                        *reinterpret_cast<u32x2*>(to) =
                            u32x2{pack_bf16(acc[i][j][0], acc[i][j][1]), pack_bf16(acc[i][j][2], acc[i][j][3])};
                }
        }
        __syncthreads();
        const uint32_t tokens = p.tokens - n0 - min(p.tokens - n0, from), rows = p.rows - m0;
        if (p.rows % (16 / kSize) == 0) {
            uint8_t* const out = static_cast<uint8_t*>(y) + ((uint64_t)(n0 + from) * p.rows + m0) * kSize;
            for (uint32_t k = threadIdx.x; k < kChunks * kPass; k += T::kThreads) {
                const uint32_t n = k / kChunks, c = k % kChunks;
                if (n < tokens && c * (16 / kSize) < rows)
                    *reinterpret_cast<u32x4*>(out + (uint64_t)n * p.rows * kSize + c * 16) =
                        *reinterpret_cast<const u32x4*>(lds + n * kRow + ((c ^ (n & kTurn)) * 16));
            }
            continue;
        }
        const uint32_t count = min(rows, T::kBm);
        const auto at = [&](uint32_t n, uint32_t e) {
            return lds + n * kRow + (((e * kSize / 16) ^ (n & kTurn)) * 16) + e * kSize % 16;
        };
        const auto half = [&](uint32_t n, uint32_t e) { return (uint32_t) * reinterpret_cast<const uint16_t*>(at(n, e)); };
        constexpr uint32_t kWords = kRow / 4;   // of a token
#pragma unroll 8
        for (uint32_t k = threadIdx.x; k < kWords * kPass; k += T::kThreads) {
            const uint32_t n = k / kWords, i = k % kWords;
            const uint64_t first = (uint64_t)(n0 + from + n) * p.rows + m0;
            const uint32_t odd = kSize == 2 ? (uint32_t)first & 1u : 0, e = kSize == 2 ? 2 * i + odd : i;
            if (n < tokens && e + 4 / kSize <= count)
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(y) + (first + e) * kSize) =
                    kSize == 4 ? *reinterpret_cast<const uint32_t*>(at(n, e)) : half(n, e) | half(n, e + 1) << 16;
        }
        if (kSize == 2 && threadIdx.x < kPass && threadIdx.x < tokens) {   // what no pair has: left of the first, the last
            const uint32_t n = threadIdx.x;
            const uint64_t first = (uint64_t)(n0 + from + n) * p.rows + m0;
            const uint32_t odd = (uint32_t)first & 1u;
            uint16_t* const out = static_cast<uint16_t*>(y) + first;
            if (odd) out[0] = (uint16_t)half(n, 0);
            if ((count - odd) & 1u) out[count - 1] = (uint16_t)half(n, count - 1);
        }
    }
}

template <class T>
__global__ __launch_bounds__(T::kThreads, 2) void gemm_fp8_big_kernel(GemmParams p) {
    __shared__ __align__(16) uint8_t lds[T::kLdsBytes];
    uint32_t mt, nt;
    if (!tile_of(blockIdx.x, (p.rows + T::kBm - 1) / T::kBm, (p.tokens + T::kBn - 1) / T::kBn, mt, nt)) return;
    const uint32_t m0 = mt * T::kBm, n0 = nt * T::kBn;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t wm = wave % T::kWavesM * T::kWaveM, wn = wave / T::kWavesM * T::kWaveN;
    const uint32_t end = p.blocks;
    const Loader<T::kBm, T::kThreads> lw(p.w, p.cols, m0, p.rows);
    const Loader<T::kBn, T::kThreads> lx(p.x, p.cols, n0, p.tokens);
    const u32x4 xs_buf = buffer_words(p.xs + (uint64_t)n0 * p.blocks, min(p.tokens - n0, T::kBn) * p.blocks * 4);
    const uint32_t xs_at = lane < T::kWaveN ? (wn + lane) * p.blocks * 4 : kNoChunk;
    constant_float* const ws = (constant_float*)(p.ws + (uint64_t)(min(m0 + wm, p.rows - 1) / kBlockCols) * p.blocks);
    // Start copying a stage (zeros past the last), in two parts: the tokens' codes, their scales, and the rows of the matrix
    // that a wave multiplies in its first step; and the other rows.
    const auto column_of = [&](uint32_t b) { return b < end ? b * kBlockCols : p.cols; };
    const auto start_first = [&](uint32_t stage, uint32_t b) {
        lw.template start<0, 2>(lds + stage * T::kCodeBytes, column_of(b));
        lx.start(lds + stage * T::kCodeBytes + T::kBm * 128, column_of(b));
        copy_words_to_lds(lds_address(lds) + T::kScalesAt + stage * T::kScaleBytes + wave * 256u, xs_buf,
                          b < end && lane < T::kWaveN ? xs_at + b * 4 : kNoChunk);
    };
    const auto start_second = [&](uint32_t stage, uint32_t b) {
        lw.template start<1, 2>(lds + stage * T::kCodeBytes, column_of(b));
    };
    f32x4 acc[T::kMi][T::kNi];
#pragma unroll
    for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) acc[i][j] = (f32x4)(0.0f);

    // The two waves of each SIMD take turns: waves 4..7 run half a step behind waves 0..3, so that one group reads
    // its fragments while the other one's products keep the matrix cores busy.  Every wave passes the same
    // barriers: the late group has one more at the start, the other one at the end.
    //   waves 0..3   read b,0   multiply b,0   read b,1     multiply b,1   read b+1,0
    //   waves 4..7              read b,0       multiply b,0 read b,1       multiply b,1
    // A half of a stage is copied as soon as both groups have read what stands in its place (a group's reads have
    // returned before the barrier behind them): what is read in b,0 gives way to that of b + 2 in b,1, what is read
    // in b,1 to that of b + 2 in b + 1,0.  So a copy has five of a stage's four turns to land in, with two stages of
    // LDS; from memory it takes about 1 us, as long as three of them.  (Whole stages, two to three turns: 1846 us at
    // 8192 tokens x 28672 x 8192; without any copies 1326.)
    constexpr uint32_t kSteps = 2, kPer = T::kMi / kSteps, kAway = 4;
    static_assert(T::kMi == 8 && T::kNi == 4 && T::kStages == 2 && T::kThreads == 512, "steps of two groups of waves");
    static_assert(lw.kLoads == 4 && lw.kRows == kPer * 16 && T::kWaveM == 2 * kPer * 16,
                  "rounds of the matrix's copies are of the first and the second step in turn");
    constexpr uint32_t kOnTheirWay = lw.kLoads + lx.kLoads + 1;   // of both halves
    const bool late = wave >= 4;
    start_first(0, 0);
    start_second(0, 0);
    start_first(1, 1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kOnTheirWay) : "memory");
    __builtin_amdgcn_s_barrier();
    if (late) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // a product takes the place of the one 4 before it, which is added to the results while the products in between
    // keep the matrix core busy (before the very first ones: zeros)
    f32x4 d[kAway];
    float s[T::kNi], last[T::kNi];
#pragma unroll
    for (uint32_t i = 0; i < kAway; ++i) d[i] = (f32x4)(0.0f);
#pragma unroll
    for (uint32_t j = 0; j < T::kNi; ++j) s[j] = 0.0f;
    const auto add = [&](uint32_t product, const float (&by)[T::kNi]) {
        f32x4& to = acc[product / T::kNi][product % T::kNi];
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) to[e] = __builtin_fmaf(d[product % kAway][e], by[product % T::kNi], to[e]);
    };
    constexpr uint32_t kProducts = T::kMi * T::kNi;
    float scale = ws[0];
    uint32_t at = 0;
    // where the lane reads: the two chunks of its rows of the matrix and of the tokens, and the scales; a stage's are
    // the other one's with one bit changed
    static_assert(T::kCodeBytes == 65536, "one bit");
    const Places places_w(wm), places_x(T::kBm + wn);
    uint32_t from_w = places_w.lo, from_w4 = places_w.hi, from_x = places_x.lo, from_x4 = places_x.hi;
    for (uint32_t b = 0; b < end; ++b, at ^= 1) {
        const float* const sc = reinterpret_cast<const float*>(lds + T::kScalesAt + at * T::kScaleBytes) + wave * 64;
        i32x8 x[T::kNi];
#pragma unroll
        for (uint32_t step = 0; step < kSteps; ++step) {
            i32x8 w[kPer];
            float own[T::kNi];
#pragma unroll
            for (uint32_t i = 0; i < kPer; ++i)
                w[i] = joined(lds + from_w + (step * kPer + i) * 2048, lds + from_w4 + (step * kPer + i) * 2048);
            if (step == 0) {
#pragma unroll
                for (uint32_t j = 0; j < T::kNi; ++j) x[j] = joined(lds + from_x + j * 2048, lds + from_x4 + j * 2048);
#pragma unroll
                for (uint32_t j = 0; j < T::kNi; ++j) own[j] = sc[j * 16 + (lane & 15u)];
            }
            __builtin_amdgcn_sched_barrier(0);
            if (step == 0) {
                start_second(at ^ 1, b + 1);
            } else {
                start_first(at, b + 2);
                from_w ^= T::kCodeBytes, from_w4 ^= T::kCodeBytes, from_x ^= T::kCodeBytes, from_x4 ^= T::kCodeBytes;
            }
            __builtin_amdgcn_sched_barrier(0);
            // of the copies, those that were started in this turn and the one before may be on their way still
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kOnTheirWay) : "memory");
            if (step == 0) {
#pragma unroll
                for (uint32_t j = 0; j < T::kNi; ++j) last[j] = s[j], s[j] = own[j] * scale;
            } else {
                scale = ws[min(b + 1, end - 1)];
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t i = 0; i < kPer; ++i)
#pragma unroll
                for (uint32_t j = 0; j < T::kNi; ++j) {
                    const uint32_t product = (step * kPer + i) * T::kNi + j;
                    if (product < kAway) add(kProducts - kAway + product, last);
                    else add(product - kAway, s);
                    d[product % kAway] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[i], x[j], (f32x4)(0.0f), 0,
                                                                                         0, 0, 0, 0, 0);
                    __builtin_amdgcn_sched_group_barrier(2, 4, 0);   // four VALU instructions, then the product
                    __builtin_amdgcn_sched_group_barrier(8, 1, 0);
                }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
    }
    if (!late) __builtin_amdgcn_s_barrier();
#pragma unroll
    for (uint32_t product = kProducts - kAway; product < kProducts; ++product) add(product, s);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is on its way into LDS any more
    __syncthreads();
    store_tile<T, WC_OUT_BF16>(lds, p.y, p, m0, n0, acc);
}

// A tile whose group of waves takes every kGroups-th block of columns: a step is kGroups blocks, one barrier, and the
// groups' chains of waiting, reading and multiplying run beside each other; their sums are added in order at the end.
template <class T, bool kExact, bool kOnce>
__global__ __launch_bounds__(T::kThreads) void gemm_fp8_tile_kernel(GemmParams p) {
    __shared__ __align__(16) uint8_t lds[T::kLdsBytes];
    uint32_t mt, nt;
    if (!tile_of(blockIdx.x, (p.rows + T::kBm - 1) / T::kBm, (p.tokens + T::kBn - 1) / T::kBn, mt, nt)) return;
    const uint32_t m0 = mt * T::kBm, n0 = nt * T::kBn;
    const uint32_t all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t group = all / T::kWaves, wave = all % T::kWaves;
    const uint32_t wm = wave % T::kWavesM * T::kWaveM, wn = wave / T::kWavesM * T::kWaveN;
    const uint32_t begin = blockIdx.y * p.split_blocks, end = min(begin + p.split_blocks, p.blocks);
    const Loader<T::kBm, T::kGroupThreads> lw(p.w, p.cols, m0, p.rows);
    const Loader<T::kBn, T::kGroupThreads> lx(p.x, p.cols, n0, p.tokens);
    constexpr uint32_t kLoads = lw.kLoads + lx.kLoads + 1;   // per thread and stage
    const u32x4 xs_buf = buffer_words(p.xs + (uint64_t)n0 * p.blocks, min(p.tokens - n0, T::kBn) * p.blocks * 4);
    const uint32_t xs_at = lane < T::kWaveN ? (wn + lane) * p.blocks * 4 : kNoChunk;
    constant_float* const ws = (constant_float*)(p.ws + (uint64_t)(min(m0 + wm, p.rows - 1) / kBlockCols) * p.blocks);
    uint8_t* const codes = lds + group * T::kCodeBytes;
    uint8_t* const scales = lds + T::kScalesAt + group * T::kScaleBytes + wave * 256;
    // where the matrix is read once, in one split, tiles begin at different blocks, as few tokens' groups do (64 tokens x
    // 28672 x 8192: 48.7 us, from the first one on 54.2)
    const uint32_t turn = kOnce && p.splits == 1 ? blockIdx.x / kDies * T::kGroups % (end - begin) : 0;
    const auto turned = [&](uint32_t b) { return !kOnce || b >= end ? b : b + turn < end ? b + turn : b + turn - (end - begin); };
    const auto start = [&](uint32_t stage, uint32_t b) {   // zeros from the split's end on
        const uint32_t c0 = b < end ? turned(b) * kBlockCols : p.cols;
        uint8_t* const to = codes + stage * (T::kGroups * T::kCodeBytes);
        lw.template start<0, 1, kOnce>(to, c0);
        lx.start(to + T::kBm * 128, c0);
        copy_words_to_lds(lds_address(scales) + stage * (T::kGroups * T::kScaleBytes), xs_buf,
                          b < end && lane < T::kWaveN ? xs_at + turned(b) * 4 : kNoChunk);
    };
    f32x4 acc[T::kMi][T::kNi];
#pragma unroll
    for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) acc[i][j] = (f32x4)(0.0f);
#pragma unroll
    for (uint32_t s = 0; s + 1 < T::kStages; ++s) start(s, begin + s * T::kGroups + group);
    uint32_t at = 0, to = T::kStages - 1;
    float scale = begin + group < end ? ws[turned(begin + group)] : 0.0f;
    for (uint32_t b = begin + group; b < end + group; b += T::kGroups) {   // as often for every group
        // this stage has landed once only the later ones' copies are outstanding (each wave waits for its own, the
        // barrier joins them); past the barrier every wave is done with the stage before, which is refilled
        constexpr uint32_t kLater = (T::kStages - 2) * kLoads;
        static_assert(kLater < 64, "the load counter's range");
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLater) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        const uint8_t* const sw = codes + at * (T::kGroups * T::kCodeBytes);
        const uint8_t* const sx = sw + T::kBm * 128;
        const float* const sc = reinterpret_cast<const float*>(scales + at * (T::kGroups * T::kScaleBytes));
        i32x8 x[T::kNi], w[T::kMi];
        float s[T::kNi];
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) x[j] = fragment(sx, wn + j * 16);
#pragma unroll
        for (uint32_t i = 0; i < T::kMi; ++i) w[i] = fragment(sw, wm + i * 16);
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) s[j] = sc[j * 16 + (lane & 15u)];
        __builtin_amdgcn_sched_barrier(0);   // the reads are on their way before the copies
        start(to, b + (T::kStages - 1) * T::kGroups);
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) {
            const Operand<kExact> xj(x[j]);
            s[j] *= scale;
#pragma unroll
            for (uint32_t i = 0; i < T::kMi; ++i) {
                const f32x4 d = Operand<kExact>::product(Operand<kExact>(w[i]), xj);
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[e], s[j], acc[i][j][e]);
            }
        }
        scale = b + T::kGroups < end ? ws[turned(b + T::kGroups)] : 0.0f;
        to = at;
        at = at + 1 == T::kStages ? 0 : at + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is on its way into LDS any more
    __syncthreads();
    if constexpr (T::kGroups > 1) {   // the groups in order
        constexpr uint32_t kWaveBytes = T::kMi * T::kNi * 1024;
        static_assert((T::kGroups - 1) * T::kWaves * kWaveBytes <= T::kLdsBytes, "the other groups' sums fit");
        f32x4* const sums = reinterpret_cast<f32x4*>(lds + wave * kWaveBytes) + lane;
        constexpr uint32_t kNext = T::kWaves * kWaveBytes / 16;
        if (group)
#pragma unroll
            for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
                for (uint32_t j = 0; j < T::kNi; ++j) sums[(group - 1) * kNext + (i * T::kNi + j) * 64] = acc[i][j];
        __syncthreads();
        if (!group)
            for (uint32_t g = 0; g + 1 < T::kGroups; ++g)
#pragma unroll
                for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
                    for (uint32_t j = 0; j < T::kNi; ++j) acc[i][j] += sums[g * kNext + (i * T::kNi + j) * 64];
        __syncthreads();
    }
    if (p.splits > 1)
        store_tile<T, WC_OUT_F32>(lds, p.part + blockIdx.y * split_elems(p.tokens, p.rows), p, m0, n0, acc);
    else if (kExact && p.out_kind == WC_OUT_F32)
        store_tile<T, WC_OUT_F32>(lds, p.y, p, m0, n0, acc);
    else
        store_tile<T, WC_OUT_BF16>(lds, p.y, p, m0, n0, acc);
}

// Few tokens: up to 16 kNi, bound by reading the matrix.  A workgroup takes 16 kMi rows; its waves take blocks of columns
// in turn, each with kDepth stages of LDS of its own, so that none waits for another until the end, when their sums are
// added in order: one launch, and everything in a fixed order.  The matrix is read past the caches (1 token x 131072 x 8192:
// 170 us, through them 193, floor 167; 16 x 28672 x 8192: 48.0 and 54.4).
template <uint32_t kMi_, uint32_t kNi_, uint32_t kDepth_>
struct Few {
    static constexpr uint32_t kMi = kMi_, kNi = kNi_, kDepth = kDepth_;
    static constexpr uint32_t kCodeBytes = (kMi + kNi) * 2048, kStageBytes = kCodeBytes + 256;
    static constexpr uint32_t kWaveBytes = kDepth * kStageBytes;
    static constexpr uint32_t kLoads = (kMi + kNi) * 2 + 1;   // copies of a stage
    static_assert(kNi <= 4 && 16 * kMi <= kBlockCols && kMi * kNi * 1024 <= kWaveBytes, "shape");
};

template <class F>
__global__ __launch_bounds__(1024) void gemm_fp8_few_kernel(GemmParams p) {
    extern __shared__ __align__(16) uint8_t lds[];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t waves = blockDim.x >> 6;
    const uint32_t m0 = blockIdx.x * (16 * F::kMi);
    uint8_t* const mine = lds + wave * F::kWaveBytes;
    const uint32_t rows = min(p.rows - m0, 16 * F::kMi);
    const u32x4 w_buf = buffer_words(p.w + (uint64_t)m0 * p.cols, rows * p.cols);
    const u32x4 x_buf = buffer_words(p.x, p.tokens * p.cols);
    const u32x4 xs_buf = buffer_words(p.xs, p.tokens * p.blocks * 4);
    constant_float* const ws = (constant_float*)(p.ws + (uint64_t)(m0 / kBlockCols) * p.blocks);
    // a copy takes 8 rows of 8 chunks, laid out as in the tiles
    const uint32_t row = lane >> 3, column0 = ((lane & 7u) ^ (row / 2 & 7u)) * 16, column1 = column0 ^ 64;
    const auto start = [&](uint32_t slot, uint32_t b) {   // zeros past the last block
        uint8_t* const to = mine + slot * F::kStageBytes;
        const uint32_t c0 = b < p.blocks ? b * kBlockCols : p.cols;
#pragma unroll
        for (uint32_t half = 0; half < 2; ++half) {   // rows row and row + 8, whose chunks lie 64 bytes apart
            const uint32_t column = half ? column1 : column0, r = row + half * 8;
            const bool inside = c0 + column < p.cols;
#pragma unroll
            for (uint32_t i = 0; i < F::kMi; ++i)
                copy_once_to_lds(lds_address(to) + i * 2048 + half * 1024, w_buf,
                                 inside ? (r + i * 16) * p.cols + column : kNoChunk, min(c0, w_buf[2]));
#pragma unroll
            for (uint32_t j = 0; j < F::kNi; ++j)
                copy_to_lds(lds_address(to) + (F::kMi + j) * 2048 + half * 1024, x_buf,
                            inside ? (r + j * 16) * p.cols + column : kNoChunk, min(c0, x_buf[2]));
        }
        copy_words_to_lds(lds_address(to) + F::kCodeBytes, xs_buf,
                          b < p.blocks && lane < 16 * F::kNi ? (lane * p.blocks + b) * 4 : kNoChunk);
    };
    f32x4 acc[F::kMi][F::kNi];
#pragma unroll
    for (uint32_t i = 0; i < F::kMi; ++i)
#pragma unroll
        for (uint32_t j = 0; j < F::kNi; ++j) acc[i][j] = (f32x4)(0.0f);
    // workgroups begin at different blocks, those of one die one behind the other, so that they do not all read the same
    // columns of rows a power of two apart
    const uint32_t turn = blockIdx.x / kDies * waves % p.blocks;
    const auto turned = [&](uint32_t b) {
        return b >= p.blocks ? b : b + turn < p.blocks ? b + turn : b + turn - p.blocks;
    };
#pragma unroll
    for (uint32_t k = 0; k < F::kDepth; ++k) start(k, turned(wave + k * waves));
    uint32_t slot = 0;
    for (uint32_t b = wave; b < p.blocks; b += waves) {
        const float scale = ws[turned(b)];
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((F::kDepth - 1) * F::kLoads) : "memory");
        const uint8_t* const from = mine + slot * F::kStageBytes;
        i32x8 w[F::kMi], x[F::kNi];
        float s[F::kNi];
#pragma unroll
        for (uint32_t i = 0; i < F::kMi; ++i) w[i] = fragment(from, i * 16);
#pragma unroll
        for (uint32_t j = 0; j < F::kNi; ++j) {
            x[j] = fragment(from, (F::kMi + j) * 16);
            s[j] = reinterpret_cast<const float*>(from + F::kCodeBytes)[j * 16 + (lane & 15u)];
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read, so that the next copy may take its place
        __builtin_amdgcn_sched_barrier(0);
        start(slot, turned(b + F::kDepth * waves));
#pragma unroll
        for (uint32_t j = 0; j < F::kNi; ++j) {
            const Operand<true> xj(x[j]);
#pragma unroll
            for (uint32_t i = 0; i < F::kMi; ++i) {
                const f32x4 d = Operand<true>::product(Operand<true>(w[i]), xj);
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[e], s[j] * scale, acc[i][j][e]);
            }
        }
        slot = slot + 1 == F::kDepth ? 0 : slot + 1;
    }
    // the waves in order
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    constexpr uint32_t kOut = F::kMi * F::kNi * 256, kRows = 16 * F::kMi;   // results; rows of one token
    float* const sums = reinterpret_cast<float*>(lds);   // [wave][token][row]
#pragma unroll
    for (uint32_t j = 0; j < F::kNi; ++j)
#pragma unroll
        for (uint32_t i = 0; i < F::kMi; ++i)
            *reinterpret_cast<f32x4*>(sums + wave * kOut + (j * 16 + (lane & 15u)) * kRows + i * 16 + (lane >> 4) * 4) =
                acc[i][j];
    __syncthreads();
    for (uint32_t k = threadIdx.x * 4; k < kOut; k += blockDim.x * 4) {
        const uint32_t t = k / kRows, r = k % kRows;
        if (t >= p.tokens || r >= rows) continue;
        f32x4 v = *reinterpret_cast<const f32x4*>(sums + k);
        for (uint32_t g = 1; g < waves; ++g) v += *reinterpret_cast<const f32x4*>(sums + g * kOut + k);
        store4(p.y, p.out_kind, (uint64_t)t * p.rows + m0 + r, rows - r, v);
    }
}

// The splits' sums, in order; a split's begin on 16 bytes.
__global__ __launch_bounds__(256) void gemm_fp8_join_kernel(GemmParams p) {
    const uint64_t n = (uint64_t)p.tokens * p.rows, per = split_elems(p.tokens, p.rows);
    const uint64_t i = ((uint64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f32x4 v = *reinterpret_cast<const f32x4*>(p.part + i);
    for (uint32_t s = 1; s < p.splits; ++s) v += *reinterpret_cast<const f32x4*>(p.part + s * per + i);
    store4(p.y, p.out_kind, i, n - i < 4 ? (uint32_t)(n - i) : 4, v);
}

template <class F>
void launch_few(const GemmParams& p, uint32_t waves, hipStream_t s) {
    hipLaunchKernelGGL((gemm_fp8_few_kernel<F>), dim3(cdiv(p.rows, 16 * F::kMi)), dim3(64 * waves), waves * F::kWaveBytes, s,
                       p);
}

void launch_few_tokens(uint32_t kind, const GemmParams& p, hipStream_t s) {
    if (kind == kFew16) launch_few<Few<1, 1, 2>>(p, 8, s);
    else if (kind == kFew32) launch_few<Few<2, 1, 3>>(p, 4, s);
    else if (kind == kFew64) launch_few<Few<4, 1, 2>>(p, 4, s);
    else if (kind == kFewPairs16) launch_few<Few<1, 2, 2>>(p, 4, s);
    else launch_few<Few<2, 2, 2>>(p, 4, s);
}

template <class T, bool kExact, bool kMayBeOnce>
void launch(const GemmPlan& g, const GemmParams& p, hipStream_t s) {
    const dim3 grid(tile_grid(cdiv(p.rows, T::kBm), cdiv(p.tokens, T::kBn)), p.splits);
    if constexpr (kMayBeOnce)
        if (g.once) {
            hipLaunchKernelGGL((gemm_fp8_tile_kernel<T, kExact, true>), grid, dim3(T::kThreads), 0, s, p);
            return;
        }
    hipLaunchKernelGGL((gemm_fp8_tile_kernel<T, kExact, false>), grid, dim3(T::kThreads), 0, s, p);
}

using Big = Tile<256, 256, 2, 4, 2, 1>;

// Waves, stages and groups of each kind as they measured best.
template <bool kExact>
void launch_tiles(const GemmPlan& g, const GemmParams& p, hipStream_t s) {
    if (g.kind == 0) launch<Tile<32, 32, 2, 2, 4, 4>, kExact, false>(g, p, s);
    else if (g.kind == 1) launch<Tile<32, 64, 2, 2, 4, 2>, kExact, true>(g, p, s);
    else if (g.kind == 2) launch<Tile<64, 64, 2, 2, 3, 2>, kExact, true>(g, p, s);
    else if (g.kind == kHalf && g.pair) launch<Tile<128, 64, 4, 2, 3, 2>, kExact, true>(g, p, s);
    else if (g.kind == kHalf) launch<Tile<128, 64, 4, 2, 3, 1>, kExact, true>(g, p, s);
    else if (g.kind == kSquare) launch<Tile<128, 128, 2, kExact ? 2 : 4, kExact ? 2 : 3, 1>, kExact, !kExact>(g, p, s);
    else if (g.kind == 5) launch<Tile<256, 128, 4, 2, 3, 1>, kExact, true>(g, p, s);
    else if constexpr (!kExact)
        hipLaunchKernelGGL(gemm_fp8_big_kernel<Big>, dim3(tile_grid(cdiv(p.rows, Big::kBm), cdiv(p.tokens, Big::kBn))),
                           dim3(Big::kThreads), 0, s, p);
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wc_fp8_check(const wc_fp8_matrix* W) {
    if (!W || W->cols == 0 || W->cols % 16 != 0 || W->cols > WC_MAX_DIM || W->rows > WC_MAX_VOCAB)
        return WC_ERR_INVALID_ARG;
    if (W->rows == 0) return WC_OK;
    return aligned(W->codes, 16) && aligned(W->scales, 4) ? WC_OK : WC_ERR_INVALID_ARG;
}

extern "C" int wc_gemm_fp8_work_bytes(const wc_fp8_matrix* W, uint64_t tokens, uint64_t* work_bytes) {
    const int st = wc_fp8_check(W);
    if (st != WC_OK) return st;
    if (!work_bytes || tokens > WC_MAX_TOKENS || tokens * W->rows > WC_MAX_LOGITS) return WC_ERR_INVALID_ARG;
    *work_bytes = 0;
    if (W->rows == 0 || tokens == 0) return WC_OK;
    for (const bool exact : {false, true}) {   // results of either type
        const uint64_t need = plan_of(W->rows, W->cols, tokens, exact).work_bytes;
        *work_bytes = need > *work_bytes ? need : *work_bytes;
    }
    return WC_OK;
}

extern "C" int wc_gemm_fp8_async(const wc_fp8_matrix* W, const uint8_t* x_codes, const float* x_scales,
                                 uint64_t tokens, void* y, uint32_t out_kind, void* work_dev, uint64_t work_bytes,
                                 void* stream) {
    uint64_t need = 0;
    const int st = wc_gemm_fp8_work_bytes(W, tokens, &need);
    if (st != WC_OK) return st;
    if (out_kind != WC_OUT_F32 && out_kind != WC_OUT_BF16) return WC_ERR_INVALID_ARG;
    if (W->rows == 0 || tokens == 0) return WC_OK;
    if (!aligned(x_codes, 16) || !aligned(x_scales, 4) || !aligned(y, 16) ||
        (need && (!aligned(work_dev, 256) || work_bytes < need)))
        return WC_ERR_INVALID_ARG;
    const bool exact = out_kind == WC_OUT_F32;
    const GemmPlan g = plan_of(W->rows, W->cols, tokens, exact);
    GemmParams p{};
    p.w = W->codes, p.ws = W->scales, p.x = x_codes, p.xs = x_scales, p.y = y;
    p.part = static_cast<float*>(work_dev);
    p.rows = W->rows, p.cols = W->cols, p.tokens = (uint32_t)tokens, p.blocks = cdiv(W->cols, kBlockCols);
    p.split_blocks = g.split_blocks, p.splits = g.splits, p.out_kind = out_kind;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (g.few) launch_few_tokens(g.kind, p, s);
    else if (exact) launch_tiles<true>(g, p, s);
    else launch_tiles<false>(g, p, s);
    if (g.splits > 1) {
        const uint32_t groups = cdiv((uint64_t)p.tokens * p.rows, 1024);
        hipLaunchKernelGGL(gemm_fp8_join_kernel, dim3(groups), dim3(256), 0, s, p);
    }
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
