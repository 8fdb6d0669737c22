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
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "e4m3.h"
#include "lds_copy.h"

namespace wc {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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
    static constexpr uint32_t kLoads = R * 8 / kThreads;
    static_assert(R * 8 % kThreads == 0 && kThreads / 8 % 16 == 0, "whole rounds, all of the same place in their rows");
    const uint8_t* base;
    uint32_t bytes, cols, column;
    uint32_t off[kLoads];
    __device__ __forceinline__ Loader(const uint8_t* p, uint32_t cols_, uint32_t row0, uint32_t rows) : cols(cols_) {   // row0 < rows
        base = p + (uint64_t)row0 * cols;
        bytes = (rows - row0 < R ? rows - row0 : R) * cols;
        const uint32_t row = threadIdx.x / 8;
        column = ((threadIdx.x & 7u) ^ (row / 2 & 7u)) * 16;
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i) off[i] = (row + i * (kThreads / 8)) * cols + column;
    }
    // Start copying the stage of columns c0 .. c0 + 127 (zeros past the last).
    __device__ __forceinline__ void start(uint8_t* lds, uint32_t c0) const {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const u32x4 rsrc = buffer_words(base, bytes);
        const bool inside = c0 + column < cols;
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i)
            copy_to_lds(lds_address(lds) + (i * kThreads + wave * 64u) * 16u, rsrc, inside ? off[i] + c0 : kNoChunk);
    }
};

// Rows x .. x + 15 of a stage: lane l has row x + l % 16, chunks l / 16 and l / 16 + 4.  (Which columns a lane has is
// of no account as long as both operands agree.)
__device__ __forceinline__ i32x8 fragment(const uint8_t* lds, uint32_t x) {
    const uint32_t lane = threadIdx.x & 63u, row = x + (lane & 15u), at = row / 2 & 7u;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(lds + row * 128 + ((lane >> 4) ^ at) * 16);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(lds + row * 128 + ((lane >> 4 | 4u) ^ at) * 16);
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
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

// A workgroup's tile: kBm rows of the matrix by kBn tokens, over kWavesM x kWavesN waves.
template <uint32_t kBm_, uint32_t kBn_, uint32_t kWavesM_, uint32_t kWavesN_, uint32_t kStages_>
struct Tile {
    static constexpr uint32_t kBm = kBm_, kBn = kBn_, kWavesM = kWavesM_, kWavesN = kWavesN_, kStages = kStages_;
    static constexpr uint32_t kThreads = 64 * kWavesM * kWavesN;
    static constexpr uint32_t kWaveM = kBm / kWavesM, kWaveN = kBn / kWavesN;
    static constexpr uint32_t kMi = kWaveM / 16, kNi = kWaveN / 16;
    static constexpr uint32_t kCodeBytes = (kBm + kBn) * 128;
    static constexpr uint32_t kStageBytes = kCodeBytes + kThreads * 4;   // and 64 tokens' scales per wave
    static constexpr uint32_t kLdsBytes = kStages * kStageBytes;
    static_assert(kWaveN <= 64 && kBlockCols % kWaveM == 0 && kLdsBytes <= 160 * 1024, "shape");
};

constexpr uint32_t kDies = 8;
// Which tile a workgroup takes.  Workgroups go to the 8 dies in turn: each die gets a contiguous run of tiles (its L2
// is its own), and within a run 4 tiles of rows go with each tile of tokens, so that the tiles in work at one time
// share operands both ways.
__device__ __forceinline__ bool tile_of(uint32_t id, uint32_t ms, uint32_t ns, uint32_t& m, uint32_t& n) {
    const uint32_t total = ms * ns, per = (total + kDies - 1) / kDies, t = id % kDies * per + id / kDies;
    if (id / kDies >= per || t >= total) return false;
    constexpr uint32_t kBand = 4;
    const uint32_t band = t / (kBand * ns), left = ms - band * kBand, width = left < kBand ? left : kBand;
    const uint32_t in = t - band * kBand * ns;
    m = band * kBand + in % width;
    n = in / width;
    return true;
}
uint32_t tile_grid(uint32_t ms, uint32_t ns) { return (ms * ns + kDies - 1) / kDies * kDies; }

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

template <class T, bool kExact>
__global__ __launch_bounds__(T::kThreads) void gemm_fp8_kernel(GemmParams p) {
    __shared__ __align__(16) uint8_t lds[T::kLdsBytes];
    uint32_t mt, nt;
    if (!tile_of(blockIdx.x, (p.rows + T::kBm - 1) / T::kBm, (p.tokens + T::kBn - 1) / T::kBn, mt, nt)) return;
    const uint32_t m0 = mt * T::kBm, n0 = nt * T::kBn;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t wm = wave % T::kWavesM * T::kWaveM, wn = wave / T::kWavesM * T::kWaveN;
    const uint32_t begin = blockIdx.y * p.split_blocks, end = min(begin + p.split_blocks, p.blocks);
    const Loader<T::kBm, T::kThreads> lw(p.w, p.cols, m0, p.rows);
    const Loader<T::kBn, T::kThreads> lx(p.x, p.cols, n0, p.tokens);
    constexpr uint32_t kLoads = lw.kLoads + lx.kLoads + 1;   // per thread and stage
    const u32x4 xs_buf = buffer_words(p.xs + (uint64_t)n0 * p.blocks, min(p.tokens - n0, T::kBn) * p.blocks * 4);
    const uint32_t xs_at = lane < T::kWaveN ? (wn + lane) * p.blocks * 4 : kNoChunk;
    const float* const ws = p.ws + (uint64_t)(min(m0 + wm, p.rows - 1) / kBlockCols) * p.blocks;
    const auto start = [&](uint32_t stage, uint32_t b) {   // zeros from the split's end on
        uint8_t* const to = lds + stage * T::kStageBytes;
        const uint32_t c0 = b < end ? b * kBlockCols : p.cols;
        lw.start(to, c0);
        lx.start(to + T::kBm * 128, c0);
        copy_words_to_lds(lds_address(to) + T::kCodeBytes + wave * 256u, xs_buf,
                          b < end && lane < T::kWaveN ? xs_at + b * 4 : kNoChunk);
    };
    f32x4 acc[T::kMi][T::kNi];
#pragma unroll
    for (uint32_t i = 0; i < T::kMi; ++i)
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) acc[i][j] = (f32x4)(0.0f);

#pragma unroll
    for (uint32_t s = 0; s + 1 < T::kStages; ++s) start(s, begin + s);
    uint32_t at = 0, to = T::kStages - 1;
    for (uint32_t b = begin; b < end; ++b) {
        // this stage has landed once only the later ones' copies are outstanding (each wave waits for its own, the
        // barrier joins them); past the barrier every wave is done with the stage before, which is refilled
        constexpr uint32_t kLater = (T::kStages - 2) * kLoads;
        static_assert(kLater < 64, "the load counter's range");
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLater) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        start(to, b + T::kStages - 1);
        const uint8_t* const sw = lds + at * T::kStageBytes;
        const uint8_t* const sx = sw + T::kBm * 128;
        const float* const sc = reinterpret_cast<const float*>(sw + T::kCodeBytes) + wave * 64;
        const float scale = ws[b];
        float s[T::kNi];
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) s[j] = sc[j * 16 + (lane & 15u)] * scale;
#pragma unroll
        for (uint32_t j = 0; j < T::kNi; ++j) {
            const Operand<kExact> x(fragment(sx, wn + j * 16));
#pragma unroll
            for (uint32_t i = 0; i < T::kMi; ++i) {
                const Operand<kExact> w(fragment(sw, wm + i * 16));
                const f32x4 d = Operand<kExact>::product(w, x);
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[e], s[j], acc[i][j][e]);
            }
        }
        to = at;
        at = at + 1 == T::kStages ? 0 : at + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing is on its way into LDS any more

    void* const y = p.splits > 1 ? p.part + (uint64_t)blockIdx.y * p.tokens * p.rows : p.y;
    const uint32_t kind = p.splits > 1 ? WC_OUT_F32 : p.out_kind;
#pragma unroll
    for (uint32_t j = 0; j < T::kNi; ++j) {
        const uint32_t t = n0 + wn + j * 16 + (lane & 15u);
        if (t >= p.tokens) continue;
#pragma unroll
        for (uint32_t i = 0; i < T::kMi; ++i) {
            const uint32_t r = m0 + wm + i * 16 + (lane >> 4) * 4;
            if (r < p.rows) store4(y, kind, (uint64_t)t * p.rows + r, p.rows - r, acc[i][j]);
        }
    }
}

// The splits' sums, in order.
__global__ __launch_bounds__(256) void gemm_fp8_join_kernel(GemmParams p) {
    const uint64_t n = (uint64_t)p.tokens * p.rows;
    for (uint64_t i = ((uint64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (uint64_t)gridDim.x * 1024) {
        const uint32_t left = n - i < 4 ? (uint32_t)(n - i) : 4;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        for (uint32_t s = 0; s < p.splits; ++s)
            for (uint32_t e = 0; e < left; ++e) v[e] += p.part[s * n + i + e];
        store4(p.y, p.out_kind, i, left, v);
    }
}

uint32_t cdiv(uint64_t a, uint32_t b) { return (uint32_t)((a + b - 1) / b); }

using Mid = Tile<128, 128, 2, 2, 2>;
using Thin = Tile<128, 32, 4, 1, 4>;
constexpr uint32_t kCus = 256;

struct GemmPlan {
    bool thin;
    uint32_t splits, split_blocks;
    uint64_t work_bytes;
};
GemmPlan plan_of(uint32_t rows, uint32_t cols, uint64_t tokens) {
    GemmPlan g{};
    g.thin = tokens <= 32;
    const uint32_t blocks = cdiv(cols, kBlockCols);
    const uint64_t tiles = (uint64_t)cdiv(rows, 128) * cdiv(tokens, g.thin ? 32 : 128);
    uint32_t splits = tiles < kCus ? (uint32_t)(kCus / tiles) : 1;
    splits = splits < blocks ? splits : blocks;
    g.split_blocks = cdiv(blocks, splits);
    g.splits = cdiv(blocks, g.split_blocks);
    g.work_bytes = g.splits > 1 ? (uint64_t)g.splits * tokens * rows * 4 : 0;
    return g;
}

template <class T, bool kExact>
void launch(const GemmParams& p, hipStream_t s) {
    hipLaunchKernelGGL((gemm_fp8_kernel<T, kExact>), dim3(tile_grid(cdiv(p.rows, T::kBm), cdiv(p.tokens, T::kBn)), p.splits),
                       dim3(T::kThreads), 0, s, p);
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
    *work_bytes = W->rows && tokens ? plan_of(W->rows, W->cols, tokens).work_bytes : 0;
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
    const GemmPlan g = plan_of(W->rows, W->cols, tokens);
    GemmParams p{};
    p.w = W->codes, p.ws = W->scales, p.x = x_codes, p.xs = x_scales, p.y = y;
    p.part = static_cast<float*>(work_dev);
    p.rows = W->rows, p.cols = W->cols, p.tokens = (uint32_t)tokens, p.blocks = cdiv(W->cols, kBlockCols);
    p.split_blocks = g.split_blocks, p.splits = g.splits, p.out_kind = out_kind;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (g.thin) launch<Thin, true>(p, s);
    else if (out_kind == WC_OUT_F32) launch<Mid, true>(p, s);
    else launch<Mid, false>(p, s);
    if (g.splits > 1) {
        const uint32_t groups = cdiv((uint64_t)p.tokens * p.rows, 1024);
        hipLaunchKernelGGL(gemm_fp8_join_kernel, dim3(groups < 4096 ? groups : 4096), dim3(256), 0, s, p);
    }
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
