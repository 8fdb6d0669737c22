// cross_entropy.hip -- softmax cross entropy of the vocabulary product, and
// its gradients, without keeping the logits.
//
// With h (tokens x dim) and W (vocab x dim) in bf16, z[t][v] = h[t] . W[v]:
//   lse[t]  = log sum_v exp(z[t][v]),   loss[t] = lse[t] - z[t][target[t]],
//   d[t][v] = (exp(z[t][v] - lse[t]) - [v = target[t]]) dloss[t],
//   dh = d W,   dW = d^T h.
// A target outside [0, vocab) marks a token without a loss: its loss, and its
// rows of d, are zero.  dW takes h with such rows zero too (copied beside the
// first piece's d), as what stands there may be no number.
//
// The loss takes one matrix product whose tiles never leave the chip: each
// workgroup computes a tile of z in fp32 accumulators and leaves, per token,
// the tile's maximum and its sum of exp(z - maximum); a second kernel joins a
// token's tiles in tile order.  The gradient computes z again, a piece of the
// vocabulary at a time, and keeps that piece's d in bf16 (the matrix cores'
// input type: a relative rounding of at most 2^-8 per value, as dh and dW
// themselves are rounded) for the two products that read it.  What the target's
// own value, as a rule by far the largest of a token's d, loses to that is kept
// per token in fp32, and goes into both: its product with W[target] is added to
// dh, its product with h[t] to dW[target], whose row often has that one token
// only.  Up to 128 tokens, what all values of d lose is kept as a second bf16
// matrix and multiplied for dW (with more, it would cost a product as large as
// dW's): then a row of dW has so few tokens that the roundings of the others'
// values do not average out either.
//
// The three products run on one tile routine, out[n][m] = sum_k A(m, k) B(n, k),
// m being the contiguous index of the output: a 32 x 32 accumulator block holds
// 4 consecutive m of one n per lane, so the loss reduces over the vocabulary
// (m) mostly inside a lane and every store is of 4 neighbours.  An operand is
// stored with k contiguous, or with m (n) contiguous (then its fragments are
// read with the transposing LDS load), so nothing is transposed in memory.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "lds_copy.h"
#include "tiles.h"

namespace wc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kUnit = 64;            // splits of a sum over k begin at multiples of this

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Round to nearest even; a NaN stays a NaN.
__device__ __forceinline__ uint16_t f32_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// One operand: element (x, k) is p[x * ld + k], or p[k * ld + x] when stored
// with x contiguous; x < rows, k < depth, everything else reads as zero.  ld
// and the contiguous extent are multiples of 8.
struct Operand {
    const uint16_t* p;
    uint64_t ld;
    uint32_t rows;
    uint32_t depth;
};

// LDS image of R x kBk elements in 16-byte chunks.  k contiguous: row x has
// kBk / 8 chunks, chunk c at place c ^ place(x): one pass of a 16-byte read
// touches 16 rows, 2 (kBk = 64) or 4 (32) per turn of the 64 banks, which so lie
// in different banks (with c ^ (x & 7) half of the LDS's time was conflicts).  x contiguous: row k has R / 8
// chunks, chunk c at place c ^ ((k & 3) << 2): the 4 rows of k that a
// transposing read touches lie 64 bytes apart.
//
// The loader copies one such image per stage straight from memory to LDS
// (each lane 16 bytes; the image's permutation is applied to the source
// addresses, since a wave writes 64 consecutive chunks).  What lies outside
// the operand is an offset outside its buffer: the load leaves zeros.
template <uint32_t kBk>
__device__ __forceinline__ uint32_t place(uint32_t x) {
    static_assert(kBk == 64 || kBk == 32, "stages of 64 or 32 k");
    return kBk == 64 ? x / 2 & 7u : x / 4 & 3u;
}

template <bool kXContig, uint32_t R, uint32_t kBk, uint32_t kThreads>
struct Loader {
    static constexpr uint32_t kLoads = R * kBk / 8 / kThreads;   // per thread and stage
    static_assert(R * kBk / 8 % kThreads == 0, "whole rounds");
    static_assert(kXContig ? kThreads % (R / 8) == 0 && kThreads / (R / 8) % 4 == 0 : kThreads / (kBk / 8) % 16 == 0,
                  "a thread's chunks of one stage have the same place in their rows");
    const uint16_t* base;
    uint32_t ld, depth, bytes;
    uint32_t k;            // k contiguous: the chunk's k within a stage
    uint32_t off[kLoads];

    __device__ __forceinline__ Loader(const Operand& o, uint32_t x0) : ld((uint32_t)o.ld), depth(o.depth) {
        const uint32_t tid = threadIdx.x;
        if (kXContig) {
            base = o.p;
            bytes = 0;
            const uint32_t row = tid / (R / 8), c = (tid % (R / 8)) ^ ((row & 3u) << 2);
            k = 0;
#pragma unroll
            for (uint32_t i = 0; i < kLoads; ++i)
                off[i] = x0 + c * 8 < o.rows ? ((row + i * (kThreads / (R / 8))) * ld + x0 + c * 8) * 2 : kNoChunk;
        } else {
            const uint32_t left = o.rows > x0 ? o.rows - x0 : 0;
            base = o.p + (uint64_t)x0 * o.ld;
            bytes = (left < R ? left : R) * ld * 2;
            constexpr uint32_t kRow = kBk / 8;   // chunks
            const uint32_t row = tid / kRow, c = (tid % kRow) ^ place<kBk>(row);
            k = c * 8;
#pragma unroll
            for (uint32_t i = 0; i < kLoads; ++i) off[i] = ((row + i * (kThreads / kRow)) * ld + c * 8) * 2;
        }
    }

    // Start copying the stage of k0 .. k0 + kBk - 1 (all zeros from the operand's end on).
    __device__ __forceinline__ void start(uint16_t* lds, uint32_t k0) const {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const uint16_t* from = base;
        uint32_t len = bytes;
        if (kXContig) {
            const uint32_t left = depth > k0 ? depth - k0 : 0;
            from = base + (uint64_t)k0 * ld;
            len = (left < kBk ? left : kBk) * ld * 2;
        }
        const u32x4 rsrc = buffer_words(from, len);
        const bool inside = kXContig || k0 + k < depth;
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i) {
            const uint32_t at = kXContig ? off[i] : inside ? off[i] + k0 * 2 : kNoChunk;
            copy_to_lds(lds_address(lds) + (i * kThreads + wave * 64u) * 16u, rsrc, at);
        }
    }
};

// The fragment of rows x .. x + 31, k .. k + 15 of a stage: lane l holds row
// x + l % 32, k + 8 (l / 32) .. + 7.
template <bool kXContig, uint32_t R, uint32_t kBk>
__device__ __forceinline__ bf16x8 fragment(const uint16_t* lds, uint32_t x, uint32_t k) {
    const uint32_t lane = threadIdx.x & 63u;
    if (!kXContig) {
        const uint32_t row = x + (lane & 31u), c = (k / 8 + (lane >> 5)) ^ place<kBk>(row);
        return *reinterpret_cast<const bf16x8*>(lds + row * kBk + c * 8);
    }
    // 16 lanes read a block of 4 k by 16 x (lane i: row k + i / 4, x + 4 (i % 4)) and receive it transposed
    // (lane i: x + i, 4 values of k)
    const uint32_t i = lane & 15u, xb = x + ((lane >> 4) & 1u) * 16u + (i & 3u) * 4u;
    const uint32_t kr = k + (lane >> 5) * 8u + (i >> 2);
    const uint32_t at = kr * R + (((xb / 8) ^ ((kr & 3u) << 2)) * 8) + (xb & 7u);
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at + 4 * R));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A workgroup's tile: kBm x kBn outputs over kWavesM x kWavesN waves, operands
// through kStages stages of LDS: while one is multiplied, the next kStages - 1
// are on their way.
//
// What bounds a large product is the matrix cores: per stage of 64 k a 256 x 256
// tile takes 2048 cycles of them on each SIMD and reads 192 KB of fragments
// from LDS (1536 cycles at 128 bytes), so neither may wait for the other.
// Measured at 4096 tokens x 131072 x 4096 (z, dh, dW in TFLOP/s):
//   128 x 128, one stage, no overlap              686  805  831
//   256 x 256, two stages, 8 waves                974  813  890
//   the same, tiles dealt to dies (tile_of)      1159 1136 1133
//   waves taking turns (kAlternate)              1249 1174 1182
// 4 waves of 128 x 128 each, which read a third less LDS, reach 885: a lone
// wave per SIMD cannot cover its own LDS reads.
template <bool kAx, bool kBx, uint32_t kBm_, uint32_t kBn_, uint32_t kWavesM_, uint32_t kWavesN_, uint32_t kStages_,
          uint32_t kBk_>
struct Tile {
    static constexpr uint32_t kBm = kBm_, kBn = kBn_, kWavesM = kWavesM_, kWavesN = kWavesN_, kStages = kStages_;
    static constexpr uint32_t kBk = kBk_;
    static_assert(kUnit % kBk == 0, "splits are whole stages");
    static constexpr uint32_t kThreads = 64 * kWavesM * kWavesN;
    static constexpr uint32_t kMi = kBm / kWavesM / 32, kNi = kBn / kWavesN / 32;
    static constexpr uint32_t kStageElems = (kBm + kBn) * kBk;
    static constexpr uint32_t kLdsElems = kStages * kStageElems;
    static constexpr bool kAlternate = kThreads == 512;
    static_assert(!kAlternate || kStages == 2, "alternating waves take two stages");
    using LoadA = Loader<kAx, kBm, kBk, kThreads>;
    using LoadB = Loader<kBx, kBn, kBk, kThreads>;

    __device__ static __forceinline__ void clear(f32x16 (&acc)[kMi][kNi]) {
#pragma unroll
        for (uint32_t i = 0; i < kMi; ++i)
#pragma unroll
            for (uint32_t j = 0; j < kNi; ++j) acc[i][j] = (f32x16)(0.0f);
    }

    // acc += sum over k in [k_begin, k_end) of A(m0 + ., k) B(n0 + ., k); k_begin
    // is a multiple of kUnit, k_end one too or the operands' end.
    __device__ static __forceinline__ void product(uint16_t* lds, const Operand& A, const Operand& B, uint32_t m0,
                                                   uint32_t n0, uint32_t k_begin, uint32_t k_end,
                                                   f32x16 (&acc)[kMi][kNi]) {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const uint32_t wm = wave % kWavesM * (kBm / kWavesM), wn = wave / kWavesM * (kBn / kWavesN);
        const LoadA la(A, m0);
        const LoadB lb(B, n0);
        uint32_t next = k_begin;   // the stage to start next (past k_end: its products are not taken)
#pragma unroll
        for (uint32_t s = 0; s + 1 < kStages; ++s, next += kBk) {
            la.start(lds + s * kStageElems, next);
            lb.start(lds + s * kStageElems + kBm * kBk, next);
        }
        uint32_t at = 0, to = (kStages - 1) * kStageElems;
        if constexpr (kAlternate) {
            // The two waves of each SIMD take turns: waves 4..7 run half a step behind waves 0..3, so that one
            // group reads its fragments while the other one's products keep the matrix cores busy.  Every wave
            // passes the same barriers: the late group has one more at the start, the other one at the end.
            // Stage k0 + kBk is copied while stage k0 is multiplied, into the LDS of the stage before, which both
            // groups have read: a group's reads have returned before the barrier behind them.
            const bool late = wave >= 4;
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            if (late) __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            for (uint32_t k0 = k_begin; k0 < k_end; k0 += kBk) {
                const uint16_t* const sa = lds + at;
                const uint16_t* const sb = lds + at + kBm * kBk;
#pragma unroll
                for (uint32_t kk = 0; kk < kBk; kk += 16) {
                    bf16x8 a[kMi], b[kNi];
#pragma unroll
                    for (uint32_t i = 0; i < kMi; ++i) a[i] = fragment<kAx, kBm, kBk>(sa, wm + i * 32, kk);
#pragma unroll
                    for (uint32_t j = 0; j < kNi; ++j) b[j] = fragment<kBx, kBn, kBk>(sb, wn + j * 32, kk);
                    if (kk == 0) la.start(lds + to, next);
                    if (kk == 16) lb.start(lds + to + kBm * kBk, next);
                    if (kk + 16 == kBk) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                    for (uint32_t i = 0; i < kMi; ++i)
#pragma unroll
                        for (uint32_t j = 0; j < kNi; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_s_setprio(0);
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                }
                next += kBk;
                to = at;
                at = at + kStageElems == kLdsElems ? 0 : at + kStageElems;
            }
            if (!late) __builtin_amdgcn_s_barrier();
        } else {
            for (uint32_t k0 = k_begin; k0 < k_end; k0 += kBk) {
                // this stage has landed once only the later ones' loads are outstanding (each wave waits for its own,
                // the barrier joins them); past the barrier every wave is done with the stage before, which is refilled
                constexpr uint32_t kLater = (kStages - 2) * (LoadA::kLoads + LoadB::kLoads);
                static_assert(kLater < 64, "the load counter's range");
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLater) : "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                la.start(lds + to, next);
                lb.start(lds + to + kBm * kBk, next);
                next += kBk;
                const uint16_t* const sa = lds + at;
                const uint16_t* const sb = lds + at + kBm * kBk;
#pragma unroll
                for (uint32_t kk = 0; kk < kBk; kk += 16) {
                    bf16x8 a[kMi], b[kNi];
#pragma unroll
                    for (uint32_t i = 0; i < kMi; ++i) a[i] = fragment<kAx, kBm, kBk>(sa, wm + i * 32, kk);
#pragma unroll
                    for (uint32_t j = 0; j < kNi; ++j) b[j] = fragment<kBx, kBn, kBk>(sb, wn + j * 32, kk);
#pragma unroll
                    for (uint32_t i = 0; i < kMi; ++i)
#pragma unroll
                        for (uint32_t j = 0; j < kNi; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
                }
                to = at;
                at = at + kStageElems == kLdsElems ? 0 : at + kStageElems;
            }
        }
        // nothing is on its way into LDS any more, and every wave is done reading it
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    // The tile row of accumulator element r of block i (its column is n()).
    __device__ static __forceinline__ uint32_t m(uint32_t i, uint32_t r) {
        const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63u;
        return wave % kWavesM * (kBm / kWavesM) + i * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3u);
    }
    __device__ static __forceinline__ uint32_t n(uint32_t j) {
        const uint32_t wave = threadIdx.x >> 6;
        return wave / kWavesM * (kBn / kWavesN) + j * 32 + (threadIdx.x & 31u);
    }
};

// A tile of bf16 results, row n of them 2 kBm bytes: put together in LDS (four
// neighbours of a row per lane, its 16-byte chunks at chunk ^ n, so that the 32
// rows that a wave writes at a time lie in different banks), then written as
// whole rows.  From the registers a row's lines would be written 16 bytes at a
// time: at 16 tokens x 131072 x 4096, where writing dW is all there is to do,
// that took 441 us.  value(i, j, r): four results from r on, as two words; rows
// and columns from n_end and m_end on are left out.  LDS is free when it begins.
template <class T, class Value>
__device__ __forceinline__ void store_rows(uint16_t* lds, uint16_t* out, uint64_t ld, uint32_t m_end, uint32_t n_end,
                                           Value value) {
    constexpr uint32_t kChunks = T::kBm / 8;
    static_assert(T::kBm * T::kBn <= T::kLdsElems, "the tile fits the stages' LDS");
#pragma unroll
    for (uint32_t j = 0; j < T::kNi; ++j)
#pragma unroll
        for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
            for (uint32_t r = 0; r < 16; r += 4) {
                const uint32_t n = T::n(j), m = T::m(i, r);
                *reinterpret_cast<u32x2*>(lds + n * T::kBm + (((m / 8) ^ (n & (kChunks - 1))) * 8) + (m & 7u)) =
                    value(i, j, r);
            }
    __syncthreads();
    for (uint32_t at = threadIdx.x; at < kChunks * T::kBn; at += T::kThreads) {
        const uint32_t n = at / kChunks, c = at % kChunks;
        if (n < n_end && c * 8 < m_end)
            *reinterpret_cast<u32x4*>(out + n * ld + c * 8) =
                *reinterpret_cast<const u32x4*>(lds + n * T::kBm + ((c ^ (n & (kChunks - 1))) * 8));
    }
}

struct CeParams {
    const uint16_t* h;
    const uint16_t* W;
    const void* targets;
    uint32_t target_bytes;     // 4 or 8
    uint32_t tokens, vocab, dim;
    float* loss;
    float* lse;
    const float* dloss;
    uint16_t* dh;
    uint16_t* dW;
    // workspace
    float2* part;              // loss: per vocabulary tile and token, {maximum, sum of exp(z - maximum)}
    float* own;                // loss: the target's logit; gradient: what the target's d loses to rounding
    uint16_t* d;               // gradient: d of one piece, [token][ldd]
    uint16_t* h_own;           // gradient: h of the tokens with a loss, zeros for others
    float* dh_part;            // gradient: dh in fp32, [split][token][dim]
    uint32_t ldd;
    uint32_t rests;            // d is followed by what its values lost to rounding, laid out the same
    uint32_t piece_begin, piece_end;   // the piece's vocabulary
    uint32_t split_k;          // vocabulary per split of dh's product, a multiple of kUnit
    uint32_t splits;
    uint32_t first;            // the first piece: dh_part is written, not added to
};

// The token's target, or vocab where it has none.
__device__ __forceinline__ uint32_t target_of(const CeParams& p, uint32_t t) {
    const int64_t v = p.target_bytes == 8 ? static_cast<const int64_t*>(p.targets)[t]
                                          : (int64_t) static_cast<const int32_t*>(p.targets)[t];
    return v >= 0 && v < (int64_t)p.vocab ? (uint32_t)v : p.vocab;
}

template <class T>
__global__ __launch_bounds__(T::kThreads) void ce_loss_kernel(CeParams p) {
    __shared__ __align__(16) uint16_t lds[T::kLdsElems];
    uint32_t tile, nt;
    if (!tile_of(blockIdx.x, (p.vocab + T::kBm - 1) / T::kBm, (p.tokens + T::kBn - 1) / T::kBn, tile, nt)) return;
    const uint32_t m0 = tile * T::kBm, n0 = nt * T::kBn;
    const Operand A{p.W, p.dim, p.vocab, p.dim}, B{p.h, p.dim, p.tokens, p.dim};
    f32x16 acc[T::kMi][T::kNi];
    T::clear(acc);
    T::product(lds, A, B, m0, n0, 0, p.dim, acc);

    float2* const seen = reinterpret_cast<float2*>(lds);   // [kWavesM][kBn]
    const uint32_t wave_m = (threadIdx.x >> 6) % T::kWavesM;
#pragma unroll
    for (uint32_t j = 0; j < T::kNi; ++j) {
        const uint32_t n = T::n(j), t = n0 + n;
        const uint32_t own = t < p.tokens ? target_of(p, t) : p.vocab;
        float top = -INFINITY;
#pragma unroll
        for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
            for (uint32_t r = 0; r < 16; ++r) {
                const uint32_t v = m0 + T::m(i, r);
                const float z = v < p.vocab ? acc[i][j][r] : -INFINITY;
                acc[i][j][r] = z;
                if (v == own && v < p.vocab) p.own[t] = z;
                // a NaN must not be lost in a maximum: it stays in the sum
                top = fmaxf(top, z);
            }
        top = fmaxf(top, __shfl_xor(top, 32));
        float sum = 0.0f;
        const float from = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
            for (uint32_t r = 0; r < 16; ++r) sum += __expf(acc[i][j][r] - from);
        sum += __shfl_xor(sum, 32);
        if ((threadIdx.x & 32u) == 0) seen[wave_m * T::kBn + n] = make_float2(top, sum);
    }
    __syncthreads();
    for (uint32_t n = threadIdx.x; n < T::kBn; n += T::kThreads) {
        if (n0 + n >= p.tokens) continue;
        float2 a = seen[n];
#pragma unroll
        for (uint32_t w = 1; w < T::kWavesM; ++w) {
            const float2 b = seen[w * T::kBn + n];
            const float top = fmaxf(a.x, b.x), from = top == -INFINITY ? 0.0f : top;
            a = make_float2(top, a.y * __expf(a.x - from) + b.y * __expf(b.x - from));
        }
        p.part[(uint64_t)tile * p.tokens + n0 + n] = a;
    }
}

constexpr uint32_t kJoinTokens = 4, kJoinLanes = 64;   // tokens per workgroup, threads per token

// Joins a token's tiles: 64 threads take the tiles in turn, then their results in order.
__global__ __launch_bounds__(kJoinTokens* kJoinLanes) void ce_join_kernel(CeParams p, uint32_t tiles) {
    const uint32_t t = blockIdx.x * kJoinTokens + threadIdx.x % kJoinTokens, lane = threadIdx.x / kJoinTokens;
    __shared__ float2 seen[kJoinLanes][kJoinTokens];
    float top = -INFINITY, sum = 0.0f;
    if (t < p.tokens)
        for (uint32_t i = lane; i < tiles; i += kJoinLanes) {
            const float2 b = p.part[(uint64_t)i * p.tokens + t];
            const float m = fmaxf(top, b.x), from = m == -INFINITY ? 0.0f : m;
            sum = sum * __expf(top - from) + b.y * __expf(b.x - from);
            top = m;
        }
    seen[lane][threadIdx.x % kJoinTokens] = make_float2(top, sum);
    __syncthreads();
    if (lane != 0 || t >= p.tokens) return;
    for (uint32_t w = 1; w < kJoinLanes; ++w) {
        const float2 b = seen[w][threadIdx.x];
        const float m = fmaxf(top, b.x), from = m == -INFINITY ? 0.0f : m;
        sum = sum * __expf(top - from) + b.y * __expf(b.x - from);
        top = m;
    }
    const float lse = top + logf(sum);
    p.lse[t] = lse;
    p.loss[t] = target_of(p, t) < p.vocab ? lse - p.own[t] : 0.0f;
}

// d of one piece, in bf16.
template <class T>
__global__ __launch_bounds__(T::kThreads) void ce_d_kernel(CeParams p) {
    __shared__ __align__(16) uint16_t lds[T::kLdsElems];
    uint32_t mt, nt;
    if (!tile_of(blockIdx.x, (p.piece_end - p.piece_begin + T::kBm - 1) / T::kBm, (p.tokens + T::kBn - 1) / T::kBn, mt,
                 nt))
        return;
    const uint32_t m0 = p.piece_begin + mt * T::kBm, n0 = nt * T::kBn;
    if (p.first && p.dW) {   // the tile's share of h_own
        const uint32_t chunks = p.dim / 8, count = min(T::kBn, p.tokens - n0) * chunks;
        const uint32_t step = (p.piece_end - p.piece_begin + T::kBm - 1) / T::kBm * T::kThreads;
        for (uint32_t i = mt * T::kThreads + threadIdx.x; i < count; i += step) {
            const uint64_t at = (uint64_t)n0 * chunks + i;
            u32x4 v = {0, 0, 0, 0};
            if (target_of(p, n0 + i / chunks) < p.vocab) v = reinterpret_cast<const u32x4*>(p.h)[at];
            reinterpret_cast<u32x4*>(p.h_own)[at] = v;
        }
    }
    const Operand A{p.W, p.dim, p.vocab, p.dim}, B{p.h, p.dim, p.tokens, p.dim};
    f32x16 acc[T::kMi][T::kNi];
    T::clear(acc);
    T::product(lds, A, B, m0, n0, 0, p.dim, acc);
    // per column of the lane: its token's target, upstream gradient and lse
    uint32_t own[T::kNi];
    float g[T::kNi], lse[T::kNi];
#pragma unroll
    for (uint32_t j = 0; j < T::kNi; ++j) {
        const uint32_t t = n0 + T::n(j);
        own[j] = t < p.tokens ? target_of(p, t) : p.vocab;
        g[j] = own[j] < p.vocab ? p.dloss[t] : 0.0f;
        lse[j] = t < p.tokens ? p.lse[t] : 0.0f;
    }
    const auto values = [&](uint32_t i, uint32_t j, uint32_t r, bool rest) {
        uint16_t b[4];
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
            const uint32_t v = m0 + T::m(i, r + e);
            float x = __expf(acc[i][j][r + e] - lse[j]);
            if (v == own[j]) x -= 1.0f;
            x = v < p.piece_end && own[j] < p.vocab ? x * g[j] : 0.0f;
            b[e] = f32_bf16(x);
            const float lost = (b[e] & 0x7F80u) == 0x7F80u ? 0.0f : x - bf16_f32(b[e]);   // (an infinity loses nothing)
            if (v == own[j] && v < p.piece_end) p.own[n0 + T::n(j)] = lost;
            if (rest) b[e] = f32_bf16(lost);
        }
        return u32x2{b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16};
    };
    uint16_t* const to = p.d + (uint64_t)n0 * p.ldd + mt * T::kBm;
    store_rows<T>(lds, to, p.ldd, T::kBm, p.tokens - n0,
                  [&](uint32_t i, uint32_t j, uint32_t r) { return values(i, j, r, false); });
    if constexpr (!T::kAlternate) {   // few tokens never take big tiles
        if (p.rests) {
            __syncthreads();
            store_rows<T>(lds, to + (uint64_t)p.tokens * p.ldd, p.ldd, T::kBm, p.tokens - n0,
                          [&](uint32_t i, uint32_t j, uint32_t r) { return values(i, j, r, true); });
        }
    }
}

// dh += d W over the piece, in fp32, the vocabulary in one split or a multiple of the dies.
template <class T>
__global__ __launch_bounds__(T::kThreads) void ce_dh_kernel(CeParams p) {
    __shared__ __align__(16) uint16_t lds[T::kLdsElems];
    // Eight splits (or a multiple) go to the dies, one die all tiles of a split: W and d come into one L2 each, once.
    const uint32_t ms = (p.dim + T::kBm - 1) / T::kBm, ns = (p.tokens + T::kBn - 1) / T::kBn;
    uint32_t mt, nt, split = 0;
    if (p.splits % kDies == 0) {
        const uint32_t i = blockIdx.x / kDies, tile = i % (ms * ns);
        split = blockIdx.x % kDies + i / (ms * ns) * kDies;
        mt = tile % ms, nt = tile / ms;
    } else if (!tile_of(blockIdx.x, ms, ns, mt, nt)) {
        return;
    }
    const uint32_t m0 = mt * T::kBm, n0 = nt * T::kBn;
    const uint32_t len = p.piece_end - p.piece_begin;
    const Operand A{p.W + (uint64_t)p.piece_begin * p.dim, p.dim, p.dim, len}, B{p.d, p.ldd, p.tokens, p.ldd};
    const uint32_t k_begin = split * p.split_k, k_end = min(k_begin + p.split_k, len);
    f32x16 acc[T::kMi][T::kNi];
    T::clear(acc);
    T::product(lds, A, B, m0, n0, k_begin, k_end, acc);
    float* const out = p.dh_part + (uint64_t)split * p.tokens * p.dim;
#pragma unroll
    for (uint32_t j = 0; j < T::kNi; ++j) {
        const uint32_t t = n0 + T::n(j);
        if (t >= p.tokens) continue;
#pragma unroll
        for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
            for (uint32_t r = 0; r < 16; r += 4) {
                const uint32_t m = m0 + T::m(i, r);
                if (m >= p.dim) continue;
                f32x4* const at = reinterpret_cast<f32x4*>(out + (uint64_t)t * p.dim + m);
                f32x4 v = {acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
                if (!p.first) v += *at;
                *at = v;
            }
    }
}

// acc += what the values of the targets lost in d to rounding, times h: of the
// piece's entries n0 .. n0 + kBn - 1, a product as dW's own whose k runs over
// the tokens with a target among them, in token order.  There are few (every
// token has one target, so all tiles of n together take each once), and they are
// looked for in the targets of all tokens, kScan per thread at a time: no list
// has to be made by a launch before.  The lost value is rounded to bf16 like d,
// which leaves 2^-16 of a value of d.  It takes 8 us of 270 (loss and gradients)
// at 515 tokens x 32003 x 1160, 0.17 ms of 14.0 at 4096 x 131072 x 4096.  LDS is
// free when it begins and when it ends.
template <class T>
__device__ __forceinline__ void add_lost(uint16_t* lds, const CeParams& p, uint32_t m0, uint32_t n0,
                                         f32x16 (&acc)[T::kMi][T::kNi]) {
    constexpr uint32_t kScan = 8, kWaves = T::kThreads / 64, kCounts = kScan * kWaves;
    constexpr uint32_t kChunksA = T::kBm / 8, kChunksB = T::kBn / 8;
    static_assert(kCounts <= 64, "a wave's lanes hold all counts");
    static_assert(T::kStageElems * 2 + T::kThreads * kScan * 8 + kCounts * 4 <= T::kLdsElems * 2,
                  "the list fits behind one stage");
    uint16_t* const sa = lds;
    uint16_t* const sb = lds + T::kBm * T::kBk;
    uint2* const list = reinterpret_cast<uint2*>(lds + T::kStageElems);   // {token, n | lost value << 16}
    uint32_t* const counts = reinterpret_cast<uint32_t*>(list + T::kThreads * kScan);
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wm = wave % T::kWavesM * (T::kBm / T::kWavesM), wn = wave / T::kWavesM * (T::kBn / T::kWavesN);
    const uint32_t from = p.piece_begin + n0, width = min(p.piece_end - from, T::kBn);
    const uint32_t* const targets = static_cast<const uint32_t*>(p.targets);
    const uint32_t words = p.target_bytes / 4;
    uint32_t t0 = 0;
    do {   // (a loop that might not be entered would keep the tile's sums in registers twice)
        uint32_t at[kScan], high[kScan];   // low and high words of targets
        float lost[kScan];                 // (of tokens with a target in the piece; all loads are on their way at once)
#pragma unroll
        for (uint32_t k = 0; k < kScan; ++k) {
            const uint32_t t = min(t0 + k * T::kThreads + threadIdx.x, p.tokens - 1);
            at[k] = targets[(uint64_t)t * words];
            high[k] = targets[(uint64_t)t * words + words - 1];
            lost[k] = p.own[t];
        }
        uint64_t has[kScan];
#pragma unroll
        for (uint32_t k = 0; k < kScan; ++k) {
            const bool fits = t0 + k * T::kThreads + threadIdx.x < p.tokens && (words == 1 || high[k] == 0);
            at[k] = fits && at[k] - from < width ? at[k] - from : ~0u;   // n, if the tile has it
            has[k] = __ballot(at[k] != ~0u);
            if (lane == 0) counts[k * kWaves + wave] = (uint32_t)__popcll(has[k]);
        }
        __syncthreads();
        uint32_t before = lane < kCounts ? counts[lane] : 0;   // of this and the counts before it
#pragma unroll
        for (uint32_t step = 1; step < 64; step *= 2) {
            const uint32_t other = (uint32_t)__shfl_up((int)before, step);
            if (lane >= step) before += other;
        }
        const uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)before, 63);
#pragma unroll
        for (uint32_t k = 0; k < kScan; ++k) {
            const uint32_t c = k * kWaves + wave;
            const uint32_t first = c ? (uint32_t)__builtin_amdgcn_readlane((int)before, c - 1) : 0;
            if (at[k] == ~0u) continue;
            const uint32_t t = t0 + k * T::kThreads + threadIdx.x;
            list[first + (uint32_t)__popcll(has[k] & ((1ull << lane) - 1))] =
                make_uint2(t, at[k] | (uint32_t)f32_bf16(lost[k]) << 16);
        }
        __syncthreads();
#pragma unroll 1
        for (uint32_t k0 = 0; k0 < total; k0 += T::kBk) {
            for (uint32_t i = threadIdx.x; i < T::kBk * kChunksA; i += T::kThreads) {
                const uint32_t row = i / kChunksA, c = i % kChunksA;
                u32x4 v = {0, 0, 0, 0};
                if (k0 + row < total && m0 + c * 8 < p.dim)
                    v = *reinterpret_cast<const u32x4*>(p.h + (uint64_t)list[k0 + row].x * p.dim + m0 + c * 8);
                *reinterpret_cast<u32x4*>(sa + row * T::kBm + (c ^ ((row & 3u) << 2)) * 8) = v;
            }
#pragma unroll 1
            for (uint32_t i = threadIdx.x; i < T::kBk * kChunksB; i += T::kThreads) {
                const uint32_t row = i / kChunksB, c = i % kChunksB;
                u32x4 v = {0, 0, 0, 0};
                const uint32_t entry = k0 + row < total ? list[k0 + row].y : 0xFFFFu;
                if ((entry & 0xFFFFu) / 8 == c) {
                    const uint32_t word = (entry >> 16) << (entry & 1u) * 16;
#pragma unroll
                    for (uint32_t e = 0; e < 4; ++e) v[e] = (entry & 7u) / 2 == e ? word : 0;
                }
                *reinterpret_cast<u32x4*>(sb + row * T::kBn + (c ^ ((row & 3u) << 2)) * 8) = v;
            }
            __syncthreads();
#pragma unroll
            for (uint32_t kk = 0; kk < T::kBk; kk += 16) {
                bf16x8 a[T::kMi], b[T::kNi];
#pragma unroll
                for (uint32_t i = 0; i < T::kMi; ++i) a[i] = fragment<true, T::kBm, T::kBk>(sa, wm + i * 32, kk);
#pragma unroll
                for (uint32_t j = 0; j < T::kNi; ++j) b[j] = fragment<true, T::kBn, T::kBk>(sb, wn + j * 32, kk);
#pragma unroll
                for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
                    for (uint32_t j = 0; j < T::kNi; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            __syncthreads();
        }
        t0 += T::kThreads * kScan;
    } while (t0 < p.tokens);
}

// dW of the piece = d^T h.  (Three workgroups of mid tiles per CU: with more
// registers, and so two, loss and gradients at 515 tokens x 32003 x 1160 take 297
// us in place of 279.)
template <class T>
__global__ __launch_bounds__(T::kThreads, T::kAlternate ? 2 : 3) void ce_dw_kernel(CeParams p) {
    __shared__ __align__(16) uint16_t lds[T::kLdsElems];
    const uint32_t len = p.piece_end - p.piece_begin;
    uint32_t mt, nt;
    if (!tile_of(blockIdx.x, (p.dim + T::kBm - 1) / T::kBm, (len + T::kBn - 1) / T::kBn, mt, nt)) return;
    const uint32_t m0 = mt * T::kBm, n0 = nt * T::kBn;
    const Operand A{p.h_own, p.dim, p.dim, p.tokens}, B{p.d, p.ldd, p.ldd, p.tokens};
    f32x16 acc[T::kMi][T::kNi];
    T::clear(acc);
    T::product(lds, A, B, m0, n0, 0, p.tokens, acc);
    if constexpr (T::kAlternate) {   // few tokens never take big tiles
        add_lost<T>(lds, p, m0, n0, acc);
    } else if (p.rests) {
        const Operand R{p.d + (uint64_t)p.tokens * p.ldd, p.ldd, p.ldd, p.tokens};
        T::product(lds, A, R, m0, n0, 0, p.tokens, acc);
    } else {
        add_lost<T>(lds, p, m0, n0, acc);
    }
    store_rows<T>(lds, p.dW + (uint64_t)(p.piece_begin + n0) * p.dim + m0, p.dim, p.dim - m0, len - n0,
                  [&](uint32_t i, uint32_t j, uint32_t r) {
                      return u32x2{f32_bf16(acc[i][j][r]) | (uint32_t)f32_bf16(acc[i][j][r + 1]) << 16,
                                   f32_bf16(acc[i][j][r + 2]) | (uint32_t)f32_bf16(acc[i][j][r + 3]) << 16};
                  });
}

// dW of no tokens.
__global__ __launch_bounds__(256) void ce_zero_kernel(uint16_t* dW, uint64_t chunks) {
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (uint64_t)gridDim.x * 256)
        reinterpret_cast<f32x4*>(dW)[i] = (f32x4)(0.0f);
}

constexpr uint32_t kRoundCols = 256 * 4;   // columns per workgroup and slice of the splits

// dh in bf16: the splits (one, or a multiple of 8), in order within each of
// kSlices of them, then the slices in order, plus what d's target value lost to
// its rounding times W[target].  One split in 8 slices left most threads idle
// (4096 x 4096: 81 us, 32 so).
template <uint32_t kSlices>
__global__ __launch_bounds__(256) void ce_dh_round_kernel(CeParams p) {
    constexpr uint32_t kLanes = 256 / kSlices;
    const uint32_t t = blockIdx.x, slice = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const uint32_t at = blockIdx.y * (kRoundCols / kSlices) + lane * 4;
    __shared__ f32x4 shared[256];
    const uint32_t per = p.splits / kSlices, begin = slice * per, end = begin + per;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (at < p.dim)
        for (uint32_t s = begin; s < end; ++s)
            v += *reinterpret_cast<const f32x4*>(p.dh_part + ((uint64_t)s * p.tokens + t) * p.dim + at);
    shared[threadIdx.x] = v;
    __syncthreads();
    if (slice != 0 || at >= p.dim) return;
#pragma unroll
    for (uint32_t k = 1; k < kSlices; ++k) v += shared[threadIdx.x + k * kLanes];
    const uint32_t own = target_of(p, t);
    if (own < p.vocab) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p.W + (uint64_t)own * p.dim + at);
        const float c = p.own[t];
        v[0] += c * __uint_as_float(w.x << 16);
        v[1] += c * __uint_as_float(w.x & 0xFFFF0000u);
        v[2] += c * __uint_as_float(w.y << 16);
        v[3] += c * __uint_as_float(w.y & 0xFFFF0000u);
    }
    const u32x2 w = {f32_bf16(v[0]) | (uint32_t)f32_bf16(v[1]) << 16, f32_bf16(v[2]) | (uint32_t)f32_bf16(v[3]) << 16};
    *reinterpret_cast<u32x2*>(p.dh + (uint64_t)t * p.dim + at) = w;
}

// The products' operands: z takes W and h with k (dim) contiguous; dh takes W^T
// with m (dim) contiguous and d with k (vocabulary) contiguous; dW takes h^T and
// d^T, the output indexes contiguous.
template <bool kAx, bool kBx>
using Big = Tile<kAx, kBx, 256, 256, 2, 4, 2, 64>;     // one workgroup per CU
template <bool kAx, bool kBx>
using Mid = Tile<kAx, kBx, 128, 128, 2, 2, 2, 64>;     // two per CU, each at 3/4 of the rate of one big one in all
template <bool kAx, bool kBx>
using MidDw = Tile<kAx, kBx, 128, 128, 2, 2, 3, 32>;   // rows of m and n either way: shorter stages, two ahead
template <bool kAx, bool kBx>
using Thin = Tile<kAx, kBx, 256, 64, 4, 1, 3, 64>;     // few tokens: bound by reading W, two stages ahead
constexpr uint32_t kThinTokens = 64;
constexpr uint32_t kCus = 256;
constexpr uint32_t kRestTokens = 128;   // up to these, what d loses is kept (see above)

// z of few tokens takes thin tiles where the vocabulary has enough of them to
// keep the memory busy (z, thin and mid, us: 16 x 131072 x 4096 190 and 204; 64
// x 5000 x 512 24 and 16).
bool takes_thin(uint64_t tokens, uint32_t vocab) { return tokens <= kThinTokens && cdiv(vocab, 256) >= kCus / 2; }

// Whether m x n outputs take big tiles: by the rounds that the card needs of
// either kind, a round of mid tiles (two per CU) taking 2/3 of one of big
// tiles.  Measured (z, big and mid, us): 515 tokens x 32003 x 1160 84 and 83;
// 1000 x 20000 x 2048 112 and 100; 200 x 100000 x 1024 81 and 90; 3000 x 4000 x
// 704 33 and 33; 4096 x 131072 x 4096 3520 and 6400.
bool takes_big(uint64_t m, uint64_t n) {
    if (m <= kRestTokens || n <= kRestTokens) return false;
    const uint64_t big = (uint64_t)cdiv(m, 256) * cdiv(n, 256), mid = (uint64_t)cdiv(m, 128) * cdiv(n, 128);
    return 3 * cdiv(big, kCus) < 2 * cdiv(mid, 2 * kCus);
}
// dh has few outputs and a long sum, which is split.  Tiles and splits are those
// that a model of the time likes best: rounds of workgroups, each with a fixed
// part and one per 64 of its sum (measured: 1.1 us in big tiles, 0.8 in mid
// ones), and the partial sums written and read once, at 4 TB/s.  One split
// per sum, or a multiple of the dies (see ce_dh_kernel).  Measured (dh, us):
// 515 tokens x 32003 x 1160 58 with the 16 splits that it takes, 94 with 10; 4 x
// 66561 x 488 12 with 128.
struct DhPlan {
    bool big;
    uint32_t splits;
};
DhPlan dh_plan(uint64_t tokens, uint32_t dim, uint64_t piece) {
    DhPlan best{};
    double best_us = 1e30;
    const struct {
        bool big;
        uint32_t edge, slots;
        double us;
    } kinds[] = {{true, 256, kCus, 1.1}, {false, 128, 2 * kCus, 0.8}};
    for (const auto& k : kinds) {
        const uint64_t tiles = (uint64_t)cdiv(dim, k.edge) * cdiv(tokens, k.edge);
        for (uint32_t s = 1; s <= 16 * kDies; s = s == 1 ? kDies : s + kDies) {
            if (s > 1 && (piece < s * kUnit || tiles * s > 4ull * k.slots)) break;
            const double units = (double)((piece + s - 1) / s) / kUnit;
            const double us = (double)((tiles * s + k.slots - 1) / k.slots) * (6.0 + units * k.us) +
                              (double)s * (double)tokens * dim * 8 / 4e6;
            if (us < best_us) best_us = us, best = {k.big, s};
        }
    }
    return best;
}
// dW: a short sum leaves the stores the most of the time, which two workgroups
// per CU overlap with products (dW, big and mid, us: 515 x 32003 x 1160 74 and
// 62; 200 x 100000 x 1024 142 and 120).
bool dw_takes_big(uint64_t tokens, uint32_t len, uint32_t dim) { return tokens >= 1024 && takes_big(dim, len); }

constexpr uint64_t kAlign = 256;
uint64_t up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

// Workspace: the loss's tile results and target logits; the gradient's d, fp32
// dh, target roundings and h of the tokens with a loss.  A piece of the vocabulary is what keeps d within
// 256 MiB, at least 1024 entries, whole tiles.
struct CeLayout {
    uint32_t piece, ldd, rests, splits, split_k;
    bool dh_big;
    uint64_t own, part, d, dh_part, h_own, loss_bytes, grad_bytes;
};

CeLayout layout(uint64_t tokens, uint32_t vocab, uint32_t dim) {
    CeLayout l{};
    const uint64_t tiles = cdiv(vocab, 128);   // the narrowest that a tile of z is
    l.own = 0;
    const uint64_t own_bytes = up(tokens * 4, kAlign);
    l.part = own_bytes;
    l.loss_bytes = l.part + up(tiles * tokens * 8, kAlign);
    l.rests = tokens <= kRestTokens;
    const uint64_t rows = tokens << l.rests;
    uint64_t piece = (256ull << 20) / (2 * rows) / 1024 * 1024;
    piece = piece < 1024 ? 1024 : piece;
    piece = piece < up(vocab, 256) ? piece : up(vocab, 256);
    l.piece = (uint32_t)piece;
    l.ldd = (uint32_t)(piece + 128);   // an odd number of 256-byte lines: neighbouring rows in different memory channels
    const DhPlan plan = dh_plan(tokens, dim, piece);
    const uint32_t splits = plan.splits;
    l.dh_big = plan.big;
    l.split_k = (uint32_t)up((piece + splits - 1) / splits, kUnit);
    l.splits = splits;   // the last ones may be empty: they leave zeros
    l.d = own_bytes;
    l.dh_part = l.d + up(rows * l.ldd * 2, kAlign);
    l.h_own = l.dh_part + up((uint64_t)l.splits * tokens * dim * 4, kAlign);
    l.grad_bytes = l.h_own + up(tokens * dim * 2, kAlign);
    return l;
}

bool sizes_fit(uint64_t tokens, uint32_t vocab, uint32_t dim) {
    return tokens <= WC_MAX_TOKENS && vocab != 0 && vocab <= WC_MAX_VOCAB && dim != 0 && dim % 8 == 0 &&
           dim <= WC_MAX_DIM && tokens * vocab <= WC_MAX_LOGITS;   // (a launch holds fewer than 2^32 threads)
}

bool aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <class T>
void run_loss(CeParams& p, hipStream_t s) {
    const uint32_t tiles = cdiv(p.vocab, T::kBm);
    hipLaunchKernelGGL(ce_loss_kernel<T>, dim3(tile_grid(tiles, cdiv(p.tokens, T::kBn))), dim3(T::kThreads), 0, s, p);
    hipLaunchKernelGGL(ce_join_kernel, dim3(cdiv(p.tokens, kJoinTokens)), dim3(kJoinTokens * kJoinLanes), 0, s, p, tiles);
}
template <class T>
void run_d(CeParams& p, hipStream_t s) {
    const uint32_t len = p.piece_end - p.piece_begin;
    hipLaunchKernelGGL(ce_d_kernel<T>, dim3(tile_grid(cdiv(len, T::kBm), cdiv(p.tokens, T::kBn))), dim3(T::kThreads), 0, s,
                       p);
}
template <class T>
void run_dh(CeParams& p, hipStream_t s) {
    const uint32_t ms = cdiv(p.dim, T::kBm), ns = cdiv(p.tokens, T::kBn);
    const dim3 grid = p.splits % kDies == 0 ? dim3(ms * ns * p.splits) : dim3(tile_grid(ms, ns));
    hipLaunchKernelGGL(ce_dh_kernel<T>, grid, dim3(T::kThreads), 0, s, p);
}
template <class T>
void run_dw(CeParams& p, hipStream_t s) {
    const uint32_t len = p.piece_end - p.piece_begin;
    hipLaunchKernelGGL(ce_dw_kernel<T>, dim3(tile_grid(cdiv(p.dim, T::kBm), cdiv(len, T::kBn))), dim3(T::kThreads), 0, s,
                       p);
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wc_ce_work_bytes(uint64_t tokens, uint32_t vocab, uint32_t dim, int grad, uint64_t* work_bytes) {
    if (!work_bytes || !sizes_fit(tokens, vocab, dim)) return WC_ERR_INVALID_ARG;
    *work_bytes = 0;
    if (tokens == 0) return WC_OK;
    const CeLayout l = layout(tokens, vocab, dim);
    *work_bytes = grad && l.grad_bytes > l.loss_bytes ? l.grad_bytes : l.loss_bytes;
    return WC_OK;
}

extern "C" int wc_ce_loss_async(const uint16_t* h, const uint16_t* W, const void* targets, uint32_t target_bytes,
                                uint64_t tokens, uint32_t vocab, uint32_t dim, float* loss, float* lse,
                                void* work_dev, uint64_t work_bytes, void* stream) {
    if (!sizes_fit(tokens, vocab, dim) || (target_bytes != 4 && target_bytes != 8)) return WC_ERR_INVALID_ARG;
    if (tokens == 0) return WC_OK;
    const CeLayout l = layout(tokens, vocab, dim);
    if (!aligned(h, 16) || !aligned(W, 16) || !aligned(targets, target_bytes) || !aligned(loss, 4) ||
        !aligned(lse, 4) || !aligned(work_dev, kAlign) || work_bytes < l.loss_bytes)
        return WC_ERR_INVALID_ARG;
    CeParams p{};
    p.h = h, p.W = W, p.targets = targets, p.target_bytes = target_bytes;
    p.tokens = (uint32_t)tokens, p.vocab = vocab, p.dim = dim;
    p.loss = loss, p.lse = lse;
    uint8_t* const w = static_cast<uint8_t*>(work_dev);
    p.own = reinterpret_cast<float*>(w + l.own);
    p.part = reinterpret_cast<float2*>(w + l.part);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (takes_thin(tokens, vocab)) run_loss<Thin<false, false>>(p, s);
    else if (takes_big(vocab, tokens)) run_loss<Big<false, false>>(p, s);
    else run_loss<Mid<false, false>>(p, s);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}

extern "C" int wc_ce_grad_async(const uint16_t* h, const uint16_t* W, const void* targets, uint32_t target_bytes,
                                uint64_t tokens, uint32_t vocab, uint32_t dim, const float* lse, const float* dloss,
                                uint16_t* dh, uint16_t* dW, void* work_dev, uint64_t work_bytes, void* stream) {
    if (!sizes_fit(tokens, vocab, dim) || (target_bytes != 4 && target_bytes != 8) || (!dh && !dW))
        return WC_ERR_INVALID_ARG;
    if (!aligned(W, 16) || (dW && !aligned(dW, 16))) return WC_ERR_INVALID_ARG;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (tokens == 0) {   // dW is zero, dh has no rows
        const uint64_t chunks = (uint64_t)vocab * dim / 8;
        if (!dW) return WC_OK;
        hipLaunchKernelGGL(ce_zero_kernel, dim3((uint32_t)(chunks < 2048 * 256 ? (chunks + 255) / 256 : 2048)), dim3(256),
                           0, s, dW, chunks);
        return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
    }
    const CeLayout l = layout(tokens, vocab, dim);
    if (!aligned(h, 16) || !aligned(targets, target_bytes) || !aligned(lse, 4) || !aligned(dloss, 4) ||
        (dh && !aligned(dh, 16)) || !aligned(work_dev, kAlign) || work_bytes < l.grad_bytes)
        return WC_ERR_INVALID_ARG;
    CeParams p{};
    p.h = h, p.W = W, p.targets = targets, p.target_bytes = target_bytes;
    p.tokens = (uint32_t)tokens, p.vocab = vocab, p.dim = dim;
    p.lse = const_cast<float*>(lse), p.dloss = dloss, p.dh = dh, p.dW = dW;
    uint8_t* const w = static_cast<uint8_t*>(work_dev);
    p.own = reinterpret_cast<float*>(w + l.own);
    p.d = reinterpret_cast<uint16_t*>(w + l.d);
    p.dh_part = reinterpret_cast<float*>(w + l.dh_part);
    p.h_own = reinterpret_cast<uint16_t*>(w + l.h_own);
    p.ldd = l.ldd, p.rests = l.rests, p.split_k = l.split_k, p.splits = l.splits;
    for (uint64_t v0 = 0; v0 < vocab; v0 += l.piece) {
        p.piece_begin = (uint32_t)v0;
        p.piece_end = (uint32_t)(v0 + l.piece < vocab ? v0 + l.piece : vocab);
        p.first = v0 == 0;
        const uint32_t len = p.piece_end - p.piece_begin;
        if (takes_thin(tokens, len)) run_d<Thin<false, false>>(p, s);
        else if (takes_big(len, tokens)) run_d<Big<false, false>>(p, s);
        else run_d<Mid<false, false>>(p, s);
        if (dh) {
            if (l.dh_big) run_dh<Big<true, false>>(p, s);
            else run_dh<Mid<true, false>>(p, s);
        }
        if (dW) {
            if (dw_takes_big(tokens, len, dim)) run_dw<Big<true, true>>(p, s);
            else run_dw<MidDw<true, true>>(p, s);
        }
    }
    if (dh && p.splits == 1)
        hipLaunchKernelGGL(ce_dh_round_kernel<1>, dim3(p.tokens, cdiv(dim, kRoundCols)), dim3(256), 0, s, p);
    else if (dh)
        hipLaunchKernelGGL(ce_dh_round_kernel<kDies>, dim3(p.tokens, cdiv(dim, kRoundCols / kDies)), dim3(256), 0, s, p);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
