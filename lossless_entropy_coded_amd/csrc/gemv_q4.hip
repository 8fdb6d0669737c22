// gemv_q4.hip -- matrix-vector products with 4-bit weights and group scales,
// the consumer of int4 code planes:
//
//   y[t][r] = sum_c scale[r][c / group] (code[r][c] - zero[r][c / group]) x[t][c]
//
// for 1..16 vectors x[t] (one token, or the few that are verified at once).
// Codes are two per byte, the first in the low nibble; zero points are 8 where
// none are given.
//
// A wave owns one row: lane l takes the 8-column chunks l, l + 64, ...,
// multiplies codes less zero point (exact in fp32) with x, sums 8 products,
// and adds them, times the group's scale, to its fp32 partial; a butterfly adds
// the lanes.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"

namespace wc {
namespace {

constexpr uint32_t kQ4Waves = 4;   // waves, and rows, per workgroup

struct Q4Params {
    const uint32_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    const uint16_t* x;
    float* y;
    uint32_t rows, cols, group, groups;
};

__global__ __launch_bounds__(64 * kQ4Waves) void gemv_q4_kernel(Q4Params p) {
    const uint32_t lane = threadIdx.x & 63u;
    const uint64_t row = (uint64_t)blockIdx.x * kQ4Waves + (threadIdx.x >> 6);
    if (row >= p.rows) return;
    const uint32_t chunks = p.cols / 8;
    const uint32_t* const w = p.codes + row * chunks;
    const uint4* const x = reinterpret_cast<const uint4*>(p.x + (uint64_t)blockIdx.y * p.cols);
    float acc = 0.0f;
    for (uint32_t c = lane; c < chunks; c += 64) {
        const uint32_t q = w[c], g = c * 8 / p.group;
        const uint4 xv = x[c];
        const float scale = __uint_as_float((uint32_t)p.scales[row * p.groups + g] << 16);
        const float zero = p.zeros ? (float)p.zeros[row * p.groups + g] : 8.0f;
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
        float sum = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            const float xi = __uint_as_float(i & 1 ? xs[i / 2] & 0xFFFF0000u : xs[i / 2] << 16);
            sum = __builtin_fmaf((float)((q >> (4 * i)) & 15u) - zero, xi, sum);
        }
        acc = __builtin_fmaf(scale, sum, acc);
    }
#pragma unroll
    for (uint32_t m = 32; m >= 1; m >>= 1) acc += __shfl_xor(acc, (int)m, 64);
    if (lane == 0) p.y[(uint64_t)blockIdx.y * p.rows + row] = acc;
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
    p.codes = reinterpret_cast<const uint32_t*>(W->codes);
    p.scales = W->scales, p.zeros = W->zeros, p.x = x, p.y = y;
    p.rows = W->rows, p.cols = W->cols, p.group = W->group;
    p.groups = (W->cols + W->group - 1) / W->group;
    hipLaunchKernelGGL(gemv_q4_kernel, dim3((W->rows + kQ4Waves - 1) / kQ4Waves, n_vecs), dim3(64 * kQ4Waves), 0,
                       static_cast<hipStream_t>(stream), p);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
