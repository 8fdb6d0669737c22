// norm.hip -- root-mean-square norm with the residual's addition, into bf16 or
// e4m3 codes with scales, and its gradient.
//
//   h = bf16(x + residual), or x;   r[t] = 1 / sqrt(mean_c h[t][c]^2 + eps);
//   y[t][c] = h[t][c] r[t] w[c];
//   with u = h r (the unit row) and g = w dy:
//   dh[t][c] = dsum[t][c] + r[t] (g[t][c] - u[t][c] mean_c(g[t][c] u[t][c])),
//   dw[c]    = sum_t dy[t][c] u[t][c].
//
// The norm is taken of the sum as it is stored, in bf16, so that the gradient,
// which reads it again, is that of what was computed.  y goes to its codes
// without being rounded to bf16 first.
//
// Both kernels read each input once and are bound by memory.  A row is held in
// registers, 8 columns per lane and round.  The gradient's workgroups take many
// rows each, sum dw over them in registers and leave one partial row; a second
// kernel adds those in order, so that results are the same bits on every run.
// Rows past the 256 MB cache are read and written past the caches (8192 x 8192
// with the residual, into codes: 78 us, 6.05 TB/s; 86 with plain loads and stores.
// 16384 x 4096: norm 87 us, 6.2 TB/s; gradient 96, 5.6 TB/s, its second kernel
// among them).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "e4m3.h"

namespace wc {
namespace {

constexpr uint32_t kMaxWaves = 16;

struct NormParams {
    const uint16_t* x;
    const uint16_t* residual;
    const uint16_t* weight;
    uint16_t* sum;
    uint16_t* y;
    uint8_t* codes;
    float* scales;
    float* rstd;
    uint32_t n, dim, blocks;
    float eps, inv_dim;
};

// The sum over the row that blockDim.x threads hold: one wave, or several, where the whole workgroup waits.  `sums` is LDS
// of kMaxWaves floats, free for the next call after one more barrier.
__device__ __forceinline__ float row_sum(float v, float* sums) {
    v = wave_sum(v);
    const uint32_t waves = blockDim.x >> 6;
    if (waves == 1) return v;
    sums += threadIdx.y * waves;
    if ((threadIdx.x & 63u) == 0) sums[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sums[0];
    for (uint32_t k = 1; k < waves; ++k) v += sums[k];
    return v;
}

template <bool kStream>
__device__ __forceinline__ u32x4 load8(const uint16_t* row, uint32_t c, uint32_t dim) {
    return c < dim ? load16<kStream>(reinterpret_cast<const u32x4*>(row + c)) : u32x4{0, 0, 0, 0};
}

// blockDim.x threads hold a row, 8 columns each in kRounds rounds; blockDim.y rows (one, unless a row is one wave).
template <uint32_t kRounds, bool kCodes, bool kStream>
__global__ __launch_bounds__(64 * kMaxWaves) void rms_norm_kernel(NormParams p) {
    __shared__ float sums[kMaxWaves];
    const uint32_t row = __builtin_amdgcn_readfirstlane(blockIdx.x * blockDim.y + threadIdx.y);
    const uint32_t dim = row < p.n ? p.dim : 0;   // past the last row, nothing is read or written: others may wait
    const uint64_t first = (uint64_t)row * p.dim;
    u32x4 h[kRounds], w[kRounds];
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * 8;
        h[k] = load8<kStream>(p.x + first, c, dim);
    }
    if (p.residual) {
        u32x4 r[kRounds];
#pragma unroll
        for (uint32_t k = 0; k < kRounds; ++k) {
            const uint32_t c = (k * blockDim.x + threadIdx.x) * 8;
            r[k] = load8<kStream>(p.residual + first, c, dim);
        }
#pragma unroll
        for (uint32_t k = 0; k < kRounds; ++k) {
            const uint32_t c = (k * blockDim.x + threadIdx.x) * 8;
            float a[8], b[8];
            unpack_bf16(h[k], a);
            unpack_bf16(r[k], b);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) a[i] += b[i];
            h[k] = pack_bf16(a);
            if (c < dim) store16<kStream>(reinterpret_cast<u32x4*>(p.sum + first + c), h[k]);
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) w[k] = load8<false>(p.weight, (k * blockDim.x + threadIdx.x) * 8, p.dim);
    float squares = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        float a[8];
        unpack_bf16(h[k], a);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) squares = __builtin_fmaf(a[i], a[i], squares);
    }
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(row_sum(squares, sums), p.inv_dim, p.eps));
    if (p.rstd && threadIdx.x == 0 && row < p.n) p.rstd[row] = rstd;
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * 8;
        float y[8], g[8];
        unpack_bf16(h[k], y);
        unpack_bf16(w[k], g);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) y[i] = y[i] * rstd * g[i];
        if (p.y && c < dim) store16<kStream>(reinterpret_cast<u32x4*>(p.y + first + c), pack_bf16(y));
        if (kCodes) {
            const BlockCodes q = block_codes(y);
            if (c < dim) {
                store16<kStream>(reinterpret_cast<u32x2*>(p.codes + first + c), q.codes);
                if (threadIdx.x % kBlockLanes == 0) p.scales[(uint64_t)row * p.blocks + c / kBlockCols] = q.scale;
            }
        }
    }
}

struct NormGradParams {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* weight;
    const float* rstd;
    const uint16_t* dsum;
    uint16_t* dh;
    float* part;               // per workgroup, its sum of dy u
    uint32_t n, dim, teams;    // teams: rows in work at a time
    float inv_dim;
};

// One row's dh, by the blockDim.x threads that hold it, and each dy u to `take(round, column of 8, value)`.  Past the last
// row nothing is read or written: others of the workgroup may wait.
template <uint32_t kRounds, bool kStream, class Take>
__device__ __forceinline__ void grad_row(const NormGradParams& p, const u32x4 (&w)[kRounds], uint32_t row, float* sums,
                                         Take take) {
    const uint32_t dim = row < p.n ? p.dim : 0;
    const uint64_t first = (uint64_t)row * p.dim;
    u32x4 dy[kRounds], h[kRounds], add[kRounds];
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * 8;
        dy[k] = load8<kStream>(p.dy + first, c, dim);
        h[k] = load8<kStream>(p.h + first, c, dim);
        add[k] = p.dsum ? load8<kStream>(p.dsum + first, c, dim) : u32x4{0, 0, 0, 0};
    }
    const float rstd = row < p.n ? p.rstd[row] : 0.0f;
    float along = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        float d[8], u[8], g[8];
        unpack_bf16(dy[k], d);
        unpack_bf16(h[k], u);
        unpack_bf16(w[k], g);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            const float du = d[i] * (u[i] * rstd);
            take(k, i, du);
            along = __builtin_fmaf(du, g[i], along);
        }
    }
    if (!p.dh) return;
    along = row_sum(along, sums) * p.inv_dim;
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * 8;
        float d[8], u[8], g[8], out[8];
        unpack_bf16(dy[k], d);
        unpack_bf16(h[k], u);
        unpack_bf16(w[k], g);
        unpack_bf16(add[k], out);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            out[i] = __builtin_fmaf(rstd, __builtin_fmaf(-along, u[i] * rstd, d[i] * g[i]), out[i]);
        if (c < dim) store16<kStream>(reinterpret_cast<u32x4*>(p.dh + first + c), pack_bf16(out));
    }
}

// A team (the threads that hold a row) takes rows team, team + teams, ...; all teams take as many turns, as those of a
// workgroup may wait for each other.
template <uint32_t kRounds, bool kStream>
__global__ __launch_bounds__(64 * kMaxWaves) void rms_norm_grad_kernel(NormGradParams p) {
    extern __shared__ __align__(16) float lds[];   // dw of one team, where there are several
    __shared__ float sums[2][kMaxWaves];
    const uint32_t team = __builtin_amdgcn_readfirstlane(blockIdx.x * blockDim.y + threadIdx.y);
    u32x4 w[kRounds];
    float dw[kRounds][8];
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        w[k] = load8<false>(p.weight, (k * blockDim.x + threadIdx.x) * 8, p.dim);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) dw[k][i] = 0.0f;
    }
    uint32_t turn = 0;
    for (uint32_t from = 0; from < p.n; from += p.teams, turn ^= 1)
        grad_row<kRounds, kStream>(p, w, from + team, sums[turn],
                                   [&](uint32_t k, uint32_t i, float du) { dw[k][i] += du; });
    if (!p.part) return;
    for (uint32_t y = 1; y < blockDim.y; ++y) {   // the workgroup's teams in order
        if (threadIdx.y == y)
#pragma unroll
            for (uint32_t k = 0; k < kRounds; ++k)
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i)
                    *reinterpret_cast<f32x4*>(lds + ((k * 2 + i) * blockDim.x + threadIdx.x) * 4) =
                        f32x4{dw[k][4 * i], dw[k][4 * i + 1], dw[k][4 * i + 2], dw[k][4 * i + 3]};
        __syncthreads();
        if (threadIdx.y == 0)
#pragma unroll
            for (uint32_t k = 0; k < kRounds; ++k)
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(lds + ((k * 2 + i) * blockDim.x + threadIdx.x) * 4);
#pragma unroll
                    for (uint32_t e = 0; e < 4; ++e) dw[k][4 * i + e] += v[e];
                }
        __syncthreads();
    }
    if (threadIdx.y != 0) return;
    float* const part = p.part + (uint64_t)blockIdx.x * p.dim;
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t c = (k * blockDim.x + threadIdx.x) * 8;
        if (c >= p.dim) continue;
        *reinterpret_cast<f32x4*>(part + c) = f32x4{dw[k][0], dw[k][1], dw[k][2], dw[k][3]};
        *reinterpret_cast<f32x4*>(part + c + 4) = f32x4{dw[k][4], dw[k][5], dw[k][6], dw[k][7]};
    }
}

// Few rows: one launch.  The first workgroups take a row (or several short ones) each, the others 64 columns of dw, for
// which they read dy and h again, from the caches, 8 columns per lane and the rows in slices: each slice's sum in order,
// then the slices in order.
constexpr uint32_t kFewCols = 64;
constexpr uint32_t kAhead = 8;   // rows of a slice on their way at a time
template <uint32_t kRounds>
__global__ __launch_bounds__(64 * kMaxWaves) void rms_norm_grad_few_kernel(NormGradParams p, uint32_t row_groups, float* dw,
                                                                          int accumulate) {
    __shared__ __align__(16) float lds[64 * kMaxWaves * 8];
    if (blockIdx.x < row_groups) {
        u32x4 w[kRounds];
#pragma unroll
        for (uint32_t k = 0; k < kRounds; ++k) w[k] = load8<false>(p.weight, (k * blockDim.x + threadIdx.x) * 8, p.dim);
        const uint32_t row = __builtin_amdgcn_readfirstlane(blockIdx.x * blockDim.y + threadIdx.y);
        grad_row<kRounds, false>(p, w, row, lds, [](uint32_t, uint32_t, float) {});
        return;
    }
    const uint32_t thread = threadIdx.y * blockDim.x + threadIdx.x, slices = blockDim.x * blockDim.y / 8;
    const uint32_t lane = thread % 8, slice = thread / 8;
    const uint32_t c0 = (blockIdx.x - row_groups) * kFewCols, c = c0 + lane * 8;
    float sum[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) sum[i] = 0.0f;
    for (uint32_t from = slice; from < p.n; from += kAhead * slices) {
        u32x4 dy[kAhead], h[kAhead];
        float rstd[kAhead];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t row = from + k * slices, dim = row < p.n ? p.dim : 0;
            dy[k] = load8<false>(p.dy + (uint64_t)row * p.dim, c, dim);
            h[k] = load8<false>(p.h + (uint64_t)row * p.dim, c, dim);
            rstd[k] = row < p.n ? p.rstd[row] : 0.0f;
        }
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            float d[8], u[8];
            unpack_bf16(dy[k], d);
            unpack_bf16(h[k], u);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) sum[i] += d[i] * (u[i] * rstd[k]);
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
        *reinterpret_cast<f32x4*>(lds + thread * 8 + i * 4) =
            f32x4{sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]};
    __syncthreads();
    if (thread >= kFewCols || c0 + thread >= p.dim) return;
    float v = lds[thread];
    for (uint32_t k = 1; k < slices; ++k) v += lds[k * kFewCols + thread];
    dw[c0 + thread] = accumulate ? dw[c0 + thread] + v : v;
}

constexpr uint32_t kJoinLanes = 8, kJoinSlices = 64;   // 4 columns per lane

// dw: the partial rows of each slice in order, then the slices in order.
__global__ __launch_bounds__(kJoinLanes * kJoinSlices) void rms_norm_join_kernel(const float* part, uint32_t parts,
                                                                               uint32_t dim, float* dw,
                                                                               int accumulate) {
    __shared__ f32x4 shared[kJoinLanes * kJoinSlices];
    const uint32_t lane = threadIdx.x % kJoinLanes, slice = threadIdx.x / kJoinLanes;
    const uint32_t c = (blockIdx.x * kJoinLanes + lane) * 4;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t per = (parts + kJoinSlices - 1) / kJoinSlices, begin = slice * per;
    const uint32_t end = begin + per < parts ? begin + per : parts;
    if (c < dim)
#pragma unroll 8
        for (uint32_t k = begin; k < end; ++k) v += *reinterpret_cast<const f32x4*>(part + (uint64_t)k * dim + c);
    shared[threadIdx.x] = v;
    __syncthreads();
    if (slice != 0 || c >= dim) return;
    for (uint32_t k = 1; k < kJoinSlices; ++k) v += shared[k * kJoinLanes + lane];
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) dw[c + e] = accumulate ? dw[c + e] + v[e] : v[e];
}

uint32_t cdiv(uint64_t a, uint32_t b) { return (uint32_t)((a + b - 1) / b); }

// How a row is held: by as many waves as take kRoundsAim rounds, up to 16 (rows past 16384 columns: in 4 or 8 rounds);
// several short rows make a workgroup of 4 waves.  Measured (us; 8 rounds, 4, 2 and, of the norm, 1):
//   norm, 8192 x 8192, codes       81.2  79.7  78.3  80.2      gradient, 16384 x 4096    114  94  96
//   norm, 16384 x 4096, bf16       90.5  89.7  87.8  86.4      gradient, 1000 x 4096    17.7  16.9  14.6
//   norm, 1 x 4096, codes           4.7   3.6   3.0   3.0      gradient, 64 x 4096       9.9  7.6  6.9
// Above 16384 columns the gradient's registers spill: 4096 x 28672 570 us, of which memory needs 146.
// 512 workgroups of the gradient each leave a partial row (16384 x 4096: 256 take 112 us, 1024 111).
constexpr uint32_t kRoundsAim = 2;
struct RowShape {
    uint32_t waves, rounds, rows;
};
RowShape row_shape(uint32_t dim) {
    const uint32_t lanes = cdiv(dim, 8);
    RowShape s{1, 1, 1};
    while (s.waves * 64 * kRoundsAim < lanes && s.waves < kMaxWaves) s.waves *= 2;
    while (s.waves * 64 * s.rounds < lanes) s.rounds *= 2;
    s.rows = s.waves < 4 ? 4 / s.waves : 1;
    return s;
}
constexpr uint32_t kGradGroups = 512;
// Up to so many rows the gradient is one launch (us, in two and in one, with dweight): 64 x 4096 7.0 and 3.6, 512 x 2048
// 9.6 and 6.8, 512 x 8192 19.0 and 12.1, 1000 x 4096 15.3 and 13.5, 1024 x 1024 9.5 and 10.0; a launch costs its caller 3.
constexpr uint64_t kFewRows = 1024;
uint32_t grad_groups(uint64_t n, const RowShape& s) {
    const uint32_t groups = cdiv(n, s.rows);
    return groups < kGradGroups ? groups : kGradGroups;
}

bool sizes_fit(uint64_t n, uint32_t dim) {
    return n <= WC_MAX_TOKENS && dim != 0 && dim % 8 == 0 && dim <= WC_MAX_DIM;
}

template <uint32_t kRounds>
void launch_norm(const NormParams& p, const RowShape& r, hipStream_t s) {
    const dim3 grid(cdiv(p.n, r.rows)), block(64 * r.waves, r.rows);
    const bool streams = (uint64_t)p.n * p.dim * (2 + (p.residual ? 4 : 0) + (p.y ? 2 : 0) + (p.codes ? 1 : 0)) > kCacheBytes;
    const auto kernel = p.codes ? (streams ? rms_norm_kernel<kRounds, true, true> : rms_norm_kernel<kRounds, true, false>)
                                : (streams ? rms_norm_kernel<kRounds, false, true> : rms_norm_kernel<kRounds, false, false>);
    hipLaunchKernelGGL(kernel, grid, block, 0, s, p);
}

template <uint32_t kRounds>
void launch_grad(const NormGradParams& p, const RowShape& r, uint32_t groups, float* dweight, int accumulate, bool few,
                 hipStream_t s) {
    const dim3 block(64 * r.waves, r.rows);
    if (few) {
        const uint32_t row_groups = p.dh ? cdiv(p.n, r.rows) : 0;
        hipLaunchKernelGGL((rms_norm_grad_few_kernel<kRounds>), dim3(row_groups + cdiv(p.dim, kFewCols)), block, 0, s, p,
                           row_groups, dweight, accumulate);
        return;
    }
    const uint32_t bytes = r.rows > 1 ? r.waves * kRounds * 64 * 8 * 4 : 0;
    const bool streams = (uint64_t)p.n * p.dim * (4 + (p.dsum ? 2 : 0) + (p.dh ? 2 : 0)) > kCacheBytes;
    const auto kernel = streams ? rms_norm_grad_kernel<kRounds, true> : rms_norm_grad_kernel<kRounds, false>;
    hipLaunchKernelGGL(kernel, dim3(groups), block, bytes, s, p);
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wc_rms_norm_async(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint64_t n,
                                 uint32_t dim, float eps, uint16_t* sum, uint16_t* y, uint8_t* codes, float* scales,
                                 float* rstd, void* stream) {
    if (!sizes_fit(n, dim) || !(eps >= 0.0f)) return WC_ERR_INVALID_ARG;
    if (n == 0) return WC_OK;
    if ((!y && !codes) || (codes != nullptr) != (scales != nullptr) || (residual != nullptr) != (sum != nullptr))
        return WC_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned_or_null(residual, 16) || !aligned_or_null(sum, 16) ||
        !aligned_or_null(y, 16) || !aligned_or_null(codes, 16) || !aligned_or_null(scales, 4) ||
        !aligned_or_null(rstd, 4))
        return WC_ERR_INVALID_ARG;
    NormParams p{};
    p.x = x, p.residual = residual, p.weight = weight, p.sum = sum, p.y = y, p.codes = codes, p.scales = scales;
    p.rstd = rstd, p.n = (uint32_t)n, p.dim = dim, p.blocks = cdiv(dim, kBlockCols), p.eps = eps;
    p.inv_dim = 1.0f / (float)dim;
    const RowShape r = row_shape(dim);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (r.rounds == 1) launch_norm<1>(p, r, s);
    else if (r.rounds == 2) launch_norm<2>(p, r, s);
    else if (r.rounds == 4) launch_norm<4>(p, r, s);
    else launch_norm<8>(p, r, s);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}

extern "C" int wc_rms_norm_grad_work_bytes(uint64_t n, uint32_t dim, uint64_t* work_bytes) {
    if (!work_bytes || !sizes_fit(n, dim)) return WC_ERR_INVALID_ARG;
    *work_bytes = (uint64_t)grad_groups(n, row_shape(dim)) * dim * 4;
    return WC_OK;
}

extern "C" int wc_rms_norm_grad_async(const uint16_t* dy, const uint16_t* h, const uint16_t* weight,
                                      const float* rstd, const uint16_t* dsum, uint64_t n, uint32_t dim, uint16_t* dh,
                                      float* dweight, int accumulate, void* work_dev, uint64_t work_bytes,
                                      void* stream) {
    if (!sizes_fit(n, dim) || (n != 0 && !dh && !dweight) || !aligned_or_null(dweight, 4)) return WC_ERR_INVALID_ARG;
    if (n == 0 && (!dweight || accumulate)) return WC_OK;
    const RowShape r = row_shape(dim);
    const uint32_t groups = grad_groups(n, r);
    if (n != 0 && (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
                   !aligned_or_null(dsum, 16) || !aligned_or_null(dh, 16) ||
                   (dweight && (!aligned(work_dev, 256) || work_bytes < (uint64_t)groups * dim * 4))))
        return WC_ERR_INVALID_ARG;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    NormGradParams p{};
    // rows that are being overwritten cannot be read again
    const bool few = n != 0 && n <= kFewRows && dweight && dh != dy && dh != h;
    if (n != 0) {
        p.dy = dy, p.h = h, p.weight = weight, p.rstd = rstd, p.dsum = dsum, p.dh = dh;
        p.part = dweight ? static_cast<float*>(work_dev) : nullptr;
        p.n = (uint32_t)n, p.dim = dim, p.teams = groups * r.rows, p.inv_dim = 1.0f / (float)dim;
        if (r.rounds == 1) launch_grad<1>(p, r, groups, dweight, accumulate, few, s);
        else if (r.rounds == 2) launch_grad<2>(p, r, groups, dweight, accumulate, few, s);
        else if (r.rounds == 4) launch_grad<4>(p, r, groups, dweight, accumulate, few, s);
        else launch_grad<8>(p, r, groups, dweight, accumulate, few, s);
    }
    if (dweight && !few)   // of no tokens: zeros
        hipLaunchKernelGGL(rms_norm_join_kernel, dim3(cdiv(dim, kJoinLanes * 4)), dim3(kJoinLanes * kJoinSlices), 0, s,
                           p.part, n ? groups : 0, dim, dweight, accumulate);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
