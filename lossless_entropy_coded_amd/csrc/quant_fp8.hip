// quant_fp8.hip -- activations to e4m3 codes with a scale per 128 columns:
//
//   scale[t][b] = max over block b of |y[t][c]| / 448,   code[t][c] = e4m3(y[t][c] / scale[t][b]),
//
// y being x, or silu(gate) * up = gate / (1 + exp(-gate)) * up of an x that
// holds gate and up side by side.  y is never rounded before its code is.
//
// The kernel moves bytes: a lane takes 8 columns, so that a row of 16 lanes has
// a block and its largest value comes from four lane exchanges; a wave takes a
// part of one row, with all its loads started before the first is used.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "e4m3.h"

namespace wc {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = kThreads / 64;

struct QuantParams {
    const uint16_t* x;
    uint8_t* codes;
    float* scales;
    uint32_t waves;            // in all
    uint32_t parts;            // waves per row
    uint32_t dim, blocks;
};

// kRounds: 64 lanes of 8 columns per wave.
template <bool kGated, uint32_t kRounds>
__global__ __launch_bounds__(kThreads) void quant_fp8_kernel(QuantParams p) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
    if (wave >= p.waves) return;
    const uint32_t lane = threadIdx.x & 63u;
    const uint64_t row = wave / p.parts;
    const uint32_t c0 = wave % p.parts * (kRounds * 512) + lane * 8;
    const uint16_t* const x = p.x + row * p.dim * (kGated ? 2 : 1);
    u32x4 a[kRounds], b[kRounds];
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t c = c0 + k * 512;
        a[k] = b[k] = u32x4{0, 0, 0, 0};
        if (c < p.dim) {
            a[k] = *reinterpret_cast<const u32x4*>(x + c);
            if (kGated) b[k] = *reinterpret_cast<const u32x4*>(x + p.dim + c);
        }
    }
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t c = c0 + k * 512;
        float y[8];
        unpack_bf16(a[k], y);
        if (kGated) {
            float up[8];
            unpack_bf16(b[k], up);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) y[i] = y[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-y[i])) * up[i];
        }
        const BlockCodes q = block_codes(y);
        if (c < p.dim) {
            *reinterpret_cast<u32x2*>(p.codes + row * p.dim + c) = q.codes;
            if (lane % kBlockLanes == 0) p.scales[row * p.blocks + c / kBlockCols] = q.scale;
        }
    }
}

template <uint32_t kRounds>
void launch(QuantParams& p, uint64_t n, bool gated, hipStream_t s) {
    p.parts = (p.dim + kRounds * 512 - 1) / (kRounds * 512);
    p.waves = (uint32_t)(n * p.parts);   // below 2^28
    const dim3 grid((p.waves + kWaves - 1) / kWaves);
    if (gated) hipLaunchKernelGGL((quant_fp8_kernel<true, kRounds>), grid, dim3(kThreads), 0, s, p);
    else hipLaunchKernelGGL((quant_fp8_kernel<false, kRounds>), grid, dim3(kThreads), 0, s, p);
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wc_quant_fp8_async(const uint16_t* x, uint64_t n, uint32_t dim, int gated, uint8_t* codes,
                                  float* scales, void* stream) {
    if (n > WC_MAX_TOKENS || dim == 0 || dim % 8 != 0 || dim > WC_MAX_DIM) return WC_ERR_INVALID_ARG;
    if (n == 0) return WC_OK;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return WC_ERR_INVALID_ARG;
    QuantParams p{};
    p.x = x, p.codes = codes, p.scales = scales;
    p.dim = dim, p.blocks = (dim + kBlockCols - 1) / kBlockCols;
    launch<2>(p, n, gated != 0, static_cast<hipStream_t>(stream));
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
