// quant_fp8.hip -- activations to e4m3 codes with a scale per 128 columns:
//
//   scale[t][b] = max over block b of |y[t][c]| / 448,   code[t][c] = e4m3(y[t][c] / scale[t][b]),
//
// y being x, or silu(gate) * up = gate / (1 + exp(-gate)) * up of an x that
// holds gate and up side by side.  y is never rounded before its code is.
//
// The kernel moves bytes: a lane takes 8 columns, so that a row of 16 lanes has
// a block and its largest value comes from four lane exchanges; a wave takes 512
// columns of one row.  Rows past the 256 MB cache are read and written past the
// caches.  8192 x 28672, gated (1.18 GB), us: 182, which is the rate of a large copy
// (6.5 TB/s); 194 with two or four times 512 columns per wave; two times 512 and
// plain loads and stores: 211.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "e4m3.h"

namespace wc {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = kThreads / 64;
constexpr uint32_t kWaveCols = 512;
constexpr uint32_t kMostGroups = 1u << 22;   // a launch holds fewer than 2^32 threads: more waves than these have take turns

struct QuantParams {
    const uint16_t* x;
    uint8_t* codes;
    float* scales;
    uint32_t waves;            // in all
    uint32_t parts;            // waves per row
    uint32_t dim, blocks;
};

template <bool kGated, bool kStream>
__global__ __launch_bounds__(kThreads) void quant_fp8_kernel(QuantParams p) {
    const uint32_t lane = threadIdx.x & 63u;
    for (uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6)); wave < p.waves;
         wave += gridDim.x * kWaves) {
        const uint64_t row = wave / p.parts;
        const uint32_t c = wave % p.parts * kWaveCols + lane * 8;
        const uint16_t* const x = p.x + row * p.dim * (kGated ? 2 : 1);
        const bool inside = c < p.dim;
        u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (inside) {
            a = load16<kStream>(reinterpret_cast<const u32x4*>(x + c));
            if (kGated) b = load16<kStream>(reinterpret_cast<const u32x4*>(x + p.dim + c));
        }
        float y[8];
        unpack_bf16(a, y);
        if (kGated) {
            float up[8];
            unpack_bf16(b, up);
#pragma unroll
            for (uint32_t i = 0; i < 8; ++i) y[i] = y[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-y[i])) * up[i];
        }
        const BlockCodes q = block_codes(y);
        if (inside) {
            store16<kStream>(reinterpret_cast<u32x2*>(p.codes + row * p.dim + c), q.codes);
            if (lane % kBlockLanes == 0) p.scales[row * p.blocks + c / kBlockCols] = q.scale;
        }
    }
}

template <bool kGated, bool kStream>
void launch(QuantParams& p, uint64_t n, hipStream_t s) {
    p.parts = (p.dim + kWaveCols - 1) / kWaveCols;
    p.waves = (uint32_t)(n * p.parts);   // at most 2^27
    const uint32_t groups = (p.waves + kWaves - 1) / kWaves;
    hipLaunchKernelGGL((quant_fp8_kernel<kGated, kStream>), dim3(groups < kMostGroups ? groups : kMostGroups),
                       dim3(kThreads), 0, s, p);
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
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool streams = n * dim * (gated ? 5 : 3) > kCacheBytes;
    if (gated) streams ? launch<true, true>(p, n, s) : launch<true, false>(p, n, s);
    else streams ? launch<false, true>(p, n, s) : launch<false, false>(p, n, s);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
