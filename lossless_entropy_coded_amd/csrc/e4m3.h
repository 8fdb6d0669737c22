// e4m3.h -- bf16 words and e4m3 codes with a scale per block of 128 columns
// (gfx950): what the kernels that write or read such codes share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"

namespace wc {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kBlockCols = WC_FP8_BLOCK;
constexpr uint32_t kBlockLanes = kBlockCols / 8;   // lanes of a block, 8 columns each

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// Round to nearest even; a NaN stays a NaN.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
}
__device__ __forceinline__ void unpack_bf16(const u32x4& w, float (&f)[8]) {
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
}
__device__ __forceinline__ u32x4 pack_bf16(const float (&f)[8]) {
    return u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
}

// Loads and stores, kStream: past the caches, for what is too large to be found in them again.
constexpr uint64_t kCacheBytes = 256ull << 20;
template <bool kStream, class T>
__device__ __forceinline__ T load16(const T* p) {
    return kStream ? __builtin_nontemporal_load(p) : *p;
}
template <bool kStream, class T>
__device__ __forceinline__ void store16(T* p, const T& v) {
    if (kStream) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// The lane's value in the lane that the four DPP steps pair it with: lane ^ 1, lane ^ 2, half row mirrored, row
// mirrored.  After all four, a row of 16 lanes holds one result.
template <int kStep>
__device__ __forceinline__ uint32_t paired(uint32_t v) {
    constexpr int kControl[4] = {0xB1, 0x4E, 0x141, 0x140};
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kControl[kStep], 0xF, 0xF, true);
}
__device__ __forceinline__ float paired_sum(float v) {
    v += __uint_as_float(paired<0>(__float_as_uint(v)));
    v += __uint_as_float(paired<1>(__float_as_uint(v)));
    v += __uint_as_float(paired<2>(__float_as_uint(v)));
    v += __uint_as_float(paired<3>(__float_as_uint(v)));
    return v;
}
// The wave's sum, in every lane; always in the same order.
__device__ __forceinline__ float wave_sum(float v) {
    v = paired_sum(v);
    const uint32_t w = __float_as_uint(v);
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(w, w, false, false));
    v = __uint_as_float(a.x) + __uint_as_float(a.y);
    const uint32_t x = __float_as_uint(v);
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(x, x, false, false));
    return __uint_as_float(b.x) + __uint_as_float(b.y);
}

// Codes of a block whose 128 columns lie in a row of 16 lanes, 8 in each (lanes past the row's end hold zeros):
//   scale = max(largest |y|, 2^-100) * (1 / 448),   code = y / scale,
// each in fp32 (1 / 448 too), the quotient then rounded to e4m3 (to nearest, ties to even).
// The largest value becomes 448, the largest code, within roundings of fp32 that e4m3's absorbs, so no code overflows;
// the lower bound keeps the quotient of a block of zeros, or of values near fp32's end, finite.  Compared as words without
// their signs, infinities and NaNs are larger than any number: a block that has one gets the scale NaN, so that all its
// values are.
struct BlockCodes {
    u32x2 codes;
    float scale;
};
// y / scale, from 1 / scale rounded to nearest: the product, and what its remainder adds.  A quotient next to a border of
// two codes is on the right side of it (compared with the quotient in double precision, for every mantissa of the scale
// and each y near a border); the product alone is not, for one pair of bf16 mantissas in some thousands, and saves no time
// (8192 x 28672, gated, us: 184, and 182 so).  The remainder must not leave fp32's range: scales of at least 2^-64.  Zeros
// keep their signs.
__device__ __forceinline__ float quotient(float y, float scale, float inverse) {
    const float q = y * inverse;
    return __builtin_fmaf(-__builtin_fmaf(q, scale, -y), inverse, q);
}
__device__ __forceinline__ BlockCodes block_codes(const float (&y)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    top = max(top, paired<0>(top));
    top = max(top, paired<1>(top));
    top = max(top, paired<2>(top));
    top = max(top, paired<3>(top));
    const float largest = top < 0x7F800000u ? __uint_as_float(max(top, 0x0D800000u)) : NAN;   // 2^-100
    BlockCodes b;
    b.scale = largest * (1.0f / 448.0f);
    float v[8], scale = b.scale;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] = y[i];
    if (__any(largest < 0x1p-50f)) {   // small ones are lifted, both operands, so that remainders stay in range
        const float lift = largest < 0x1p-50f ? 0x1p60f : 1.0f;
        scale *= lift;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) v[i] *= lift;
    }
    const float inverse = 1.0f / scale;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] = quotient(v[i], scale, inverse);
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], w, true);
        b.codes[i] = (uint32_t)w;
    }
    return b;
}

inline bool aligned(const void* p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool aligned_or_null(const void* p, uintptr_t a) { return !p || aligned(p, a); }

}  // namespace wc
