// clip_grads.hip -- the global norm of a list of gradients, and their clipping:
//
//   norm = sqrt(sum over all tensors and elements of g^2),
//   out  = g * (max_norm / norm) where max_norm < norm < infinity, else g.
//
// Two passes over the gradients, both bound by memory.  The tensors' addresses
// and sizes are kernel arguments, kBatch tensors to a launch, so that a call
// needs no device memory for them and can be captured as it stands.  All tensors
// of a batch are cut into chunks of one size in bytes; a workgroup of the norm
// takes chunks block, block + grid, ... and leaves one partial sum, in double
// precision (no gradient of fp32 or bf16 overflows there, and long sums keep
// fp32's digits).  Of up to kOwnParts partial sums every workgroup of the second
// pass adds all by itself, in the same order, which is less than a launch in
// between would cost; more are added by such a launch.  The second pass takes one
// chunk per workgroup, from the last to the first: those read last by the first
// pass may still lie in the 256 MB cache.
//
// Four blocks of an 8B-shape model in bf16 (1.74 GB, read twice, written once), us:
//   2048 workgroups at a time, chunks of 64 KiB, plain loads and stores      993
//   loads and stores past the caches                                         920
//   8192 workgroups, chunks of 32 KiB                                        868
//   chunks of 16 KiB, one per workgroup of the second pass                   834
// which is 6.28 TB/s; a copy of 2 GB reaches 6.44.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"
#include "e4m3.h"

namespace wc {
namespace {

constexpr uint32_t kThreads = 256;
// Tensors per launch: 32 bytes of arguments each, which a launch copies: 24 of them cost their caller 1.3 us less than 96.
constexpr uint32_t kBatch = 96, kSmallBatch = 24;
constexpr uint32_t kGroups = 8192;         // workgroups of a norm's launch at most
constexpr uint32_t kOwnParts = 1024;
constexpr uint64_t kStreamBytes = 64u << 20;
constexpr uint32_t kMostChunks = 1u << 23;
constexpr uint32_t kMostChunk = 16384;     // bytes of a chunk
constexpr uint32_t kRounds = kMostChunk / 16 / kThreads;   // 16-byte loads per thread, all on their way

struct ClipTensor {
    const void* g;
    void* out;
    uint64_t numel;
    uint32_t first;     // its first chunk
    uint32_t kind;
};

template <uint32_t kTensors>
struct ClipParams {
    ClipTensor tensor[kTensors];
    double* part;
    uint32_t tensors, chunks, chunk_bytes;
    uint32_t part_at;   // the batch's first partial sum
    uint32_t parts;     // that the second pass adds, from `part` on
    float max_norm;
    float* norm;        // written by the first workgroup, where not NULL
};
static_assert(sizeof(ClipParams<kBatch>) <= 4096, "kernel arguments");

// The tensor of a chunk: the last one whose first chunk is not behind it.  Each lane looks at one tensor: a binary search
// would be a chain of loads.
template <class Params>
__device__ __forceinline__ uint32_t tensor_of(const Params& p, uint32_t chunk) {
    constexpr uint32_t kTensors = sizeof(p.tensor) / sizeof(p.tensor[0]);
    uint32_t found = 0;
#pragma unroll
    for (uint32_t from = 0; from < kTensors; from += 64) {
        const uint32_t i = from + (threadIdx.x & 63u);
        found += __popcll(__ballot(i < p.tensors && p.tensor[i < kTensors ? i : 0].first <= chunk));
    }
    return __builtin_amdgcn_readfirstlane(found - 1);
}

// The workgroup's sum of v, in every thread; always in the same order.
__device__ __forceinline__ double group_sum(double v) {
    __shared__ double sums[kThreads / 64];
#pragma unroll
    for (uint32_t d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63u) == 0) sums[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sums[0];
#pragma unroll
    for (uint32_t k = 1; k < kThreads / 64; ++k) v += sums[k];
    return v;
}

__device__ __forceinline__ double square(float f) { return (double)f * (double)f; }

// A chunk's elements begin, .. + count; the first `lanes` 16 bytes of them are taken whole (none, if the tensor is not
// aligned to them).
struct Chunk {
    uint64_t begin, wide;   // wide: the first of the 16 bytes, within the tensor
    uint32_t count, lanes, per_lane;
    template <class Params>
    __device__ __forceinline__ Chunk(const Params& p, const ClipTensor& t, uint32_t chunk) {
        const uint32_t size = t.kind == WC_OUT_F32 ? 4 : 2, per = p.chunk_bytes / size;
        per_lane = 16 / size;
        begin = (uint64_t)(chunk - t.first) * per;
        const uint64_t left = t.numel - begin;
        count = left < per ? (uint32_t)left : per;
        lanes = ((reinterpret_cast<uintptr_t>(t.g) | reinterpret_cast<uintptr_t>(t.out)) & 15u) == 0 ? count / per_lane : 0;
        wide = begin / per_lane;
    }
};
template <bool kStream>
__device__ __forceinline__ void load_chunk(const ClipTensor& t, const Chunk& c, u32x4 (&w)[kRounds]) {
    const u32x4* const g = static_cast<const u32x4*>(t.g) + c.wide;
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t i = threadIdx.x + k * kThreads;
        w[k] = i < c.lanes ? load16<kStream>(g + i) : u32x4{0, 0, 0, 0};
    }
}

__device__ __forceinline__ float value(const ClipTensor& t, uint64_t i) {
    return t.kind == WC_OUT_F32 ? static_cast<const float*>(t.g)[i]
                                : __uint_as_float((uint32_t) static_cast<const uint16_t*>(t.g)[i] << 16);
}

template <class Params, bool kStream>
__global__ __launch_bounds__(kThreads) void clip_norm_kernel(Params p) {
    double sum = 0.0;
    for (uint32_t chunk = blockIdx.x; chunk < p.chunks; chunk += gridDim.x) {
        const ClipTensor& t = p.tensor[tensor_of(p, chunk)];
        const Chunk c(p, t, chunk);
        u32x4 w[kRounds];
        load_chunk<kStream>(t, c, w);
#pragma unroll
        for (uint32_t k = 0; k < kRounds; ++k)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
                if (t.kind == WC_OUT_F32) sum += square(__uint_as_float(w[k][e]));
                else sum += square(bf16_lo(w[k][e])) + square(bf16_hi(w[k][e]));
            }
        for (uint32_t i = c.lanes * c.per_lane + threadIdx.x; i < c.count; i += kThreads) sum += square(value(t, c.begin + i));
    }
    sum = group_sum(sum);
    if (threadIdx.x == 0) p.part[p.part_at + blockIdx.x] = sum;
}

constexpr uint32_t kJoinThreads = 1024;
// The partial sums' sum, in a fixed order, behind them.
__global__ __launch_bounds__(kJoinThreads) void clip_join_kernel(double* part, uint32_t parts) {
    __shared__ double sums[kJoinThreads / 64];
    double v = 0.0;
    for (uint32_t i = threadIdx.x; i < parts; i += kJoinThreads) v += part[i];
#pragma unroll
    for (uint32_t d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63u) == 0) sums[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (uint32_t k = 1; k < kJoinThreads / 64; ++k) v += sums[k];
    part[parts] = v;
}

template <class Params, bool kStream>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(Params p) {
    const bool any = blockIdx.x < p.chunks;   // else: a list without elements, its norm alone
    const uint32_t chunk = any ? p.chunks - 1 - blockIdx.x : 0;
    const ClipTensor& t = p.tensor[any ? tensor_of(p, chunk) : 0];
    const Chunk c(p, t, chunk);
    u32x4 w[kRounds];
    if (!kStream && any) load_chunk<false>(t, c, w);   // beside the norm's sum; of large lists only what is needed
    double sum = 0.0;
    for (uint32_t i = threadIdx.x; i < p.parts; i += kThreads) sum += p.part[i];
    const double total = sqrt(group_sum(sum));
    const float norm = (float)total;
    if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
    const bool clips = norm > p.max_norm && norm < INFINITY;
    // a quotient below fp32's normal range, of which few bits would be left, is multiplied by in two steps
    const double quotient = (double)p.max_norm / total;
    const float last = quotient < 0x1p-100 ? 0x1p-126f : 1.0f, factor = (float)(quotient / last);
    if (!any || (!clips && t.g == t.out)) return;
    if (kStream) load_chunk<true>(t, c, w);
    u32x4* const out = static_cast<u32x4*>(t.out) + c.wide;
#pragma unroll
    for (uint32_t k = 0; k < kRounds; ++k) {
        const uint32_t i = threadIdx.x + k * kThreads;
        if (i >= c.lanes) break;
        if (clips) {
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                w[k][e] = t.kind == WC_OUT_F32
                              ? __float_as_uint(__uint_as_float(w[k][e]) * factor * last)
                              : pack_bf16(bf16_lo(w[k][e]) * factor * last, bf16_hi(w[k][e]) * factor * last);
        }
        store16<kStream>(out + i, w[k]);
    }
    for (uint32_t i = c.lanes * c.per_lane + threadIdx.x; i < c.count; i += kThreads) {
        if (t.kind == WC_OUT_F32) {
            const float v = static_cast<const float*>(t.g)[c.begin + i];
            static_cast<float*>(t.out)[c.begin + i] = clips ? v * factor * last : v;
        } else {
            const uint16_t v = static_cast<const uint16_t*>(t.g)[c.begin + i];
            static_cast<uint16_t*>(t.out)[c.begin + i] =
                clips ? (uint16_t)pack_bf16(__uint_as_float((uint32_t)v << 16) * factor * last, 0.0f) : v;
        }
    }
}

uint32_t size_of(const wc_grad& g) { return g.kind == WC_OUT_F32 ? 4 : 2; }

// A list's chunks: of few gradients small ones, so that they still are work for many workgroups.  Longer lists are read and
// written past the caches (us, with and without: 45 MB 30 and 28, 180 MB 92 and 104, 718 MB 345 and 382).
struct ClipShape {
    uint32_t chunk_bytes;
    bool stream;
};
ClipShape shape_of(const wc_grad* grads, uint32_t n) {
    uint64_t bytes = 0;
    for (uint32_t i = 0; i < n; ++i) bytes += grads[i].numel * size_of(grads[i]);
    return {bytes < (8u << 20) ? 4096u : kMostChunk, bytes > kStreamBytes};
}

// The next batch: as many tensors from `at` on as fit, but those without elements, and no more chunks than a launch's
// fewer than 2^32 threads allow (one tensor has 2^22 at most).  Returns where the one after it begins.
template <uint32_t kTensors>
uint32_t next_batch(const wc_grad* grads, uint32_t n, uint32_t at, uint32_t bytes, ClipParams<kTensors>& p) {
    p.tensors = p.chunks = 0;
    p.chunk_bytes = bytes;
    for (; at < n && p.tensors < kTensors; ++at) {
        const wc_grad& g = grads[at];
        if (g.numel == 0) continue;
        const uint64_t chunks = (g.numel * size_of(g) + bytes - 1) / bytes;
        if (p.tensors && p.chunks + chunks > kMostChunks) break;
        p.tensor[p.tensors++] = ClipTensor{g.g, g.out, g.numel, p.chunks, g.kind};
        p.chunks += (uint32_t)chunks;
    }
    return at;
}
uint32_t groups_of(uint32_t chunks) { return chunks < kGroups ? chunks : kGroups; }

bool list_fits(const wc_grad* grads, uint32_t n) {
    if (n > WC_MAX_GRADS || (n && !grads)) return false;
    for (uint32_t i = 0; i < n; ++i) {
        const wc_grad& g = grads[i];
        if (g.kind != WC_OUT_F32 && g.kind != WC_OUT_BF16) return false;
        if (g.numel > WC_MAX_GRAD_NUMEL) return false;
        if (g.numel && (!aligned(g.g, size_of(g)) || !aligned(g.out, size_of(g)))) return false;
    }
    return true;
}

// Partial sums of a list.
template <uint32_t kTensors>
uint64_t parts_of(const wc_grad* grads, uint32_t n, uint32_t bytes) {
    uint64_t parts = 0;
    ClipParams<kTensors> p{};
    for (uint32_t at = 0; at < n;) at = next_batch(grads, n, at, bytes, p), parts += groups_of(p.chunks);
    return parts;
}

template <uint32_t kTensors, bool kStream>
void run(const wc_grad* grads, uint32_t n, uint32_t bytes, float max_norm, float* norm, double* work, hipStream_t s) {
    using Params = ClipParams<kTensors>;
    Params p{};
    p.part = work;
    p.max_norm = max_norm;
    for (uint32_t at = 0; at < n;) {
        at = next_batch(grads, n, at, bytes, p);
        if (p.chunks == 0) continue;
        hipLaunchKernelGGL((clip_norm_kernel<Params, kStream>), dim3(groups_of(p.chunks)), dim3(kThreads), 0, s, p);
        p.part_at += groups_of(p.chunks);
    }
    p.parts = p.part_at;
    if (p.parts > kOwnParts) {
        hipLaunchKernelGGL(clip_join_kernel, dim3(1), dim3(kJoinThreads), 0, s, p.part, p.parts);
        p.part += p.parts;
        p.parts = 1;
    }
    p.norm = norm;
    uint32_t at = 0;
    do {   // a list without elements: its norm alone, 0
        at = next_batch(grads, n, at, bytes, p);
        if (p.chunks == 0 && !p.norm) continue;
        hipLaunchKernelGGL((clip_scale_kernel<Params, kStream>), dim3(p.chunks ? p.chunks : 1), dim3(kThreads), 0, s, p);
        p.norm = nullptr;
    } while (at < n);
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wc_clip_grads_work_bytes(const wc_grad* grads, uint32_t n, uint64_t* work_bytes) {
    if (!work_bytes || !list_fits(grads, n)) return WC_ERR_INVALID_ARG;
    const uint32_t bytes = shape_of(grads, n).chunk_bytes;
    const uint64_t parts = n <= kSmallBatch ? parts_of<kSmallBatch>(grads, n, bytes) : parts_of<kBatch>(grads, n, bytes);
    *work_bytes = parts ? (parts + 1) * sizeof(double) : 0;
    return WC_OK;
}

extern "C" int wc_clip_grads_async(const wc_grad* grads, uint32_t n, float max_norm, float* norm, void* work_dev,
                                   uint64_t work_bytes, void* stream) {
    uint64_t need = 0;
    const int st = wc_clip_grads_work_bytes(grads, n, &need);
    if (st != WC_OK) return st;
    if (!(max_norm >= 0.0f) || !aligned(norm, 4) || (need && (!aligned(work_dev, 256) || work_bytes < need)))
        return WC_ERR_INVALID_ARG;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const ClipShape shape = shape_of(grads, n);
    double* const work = static_cast<double*>(work_dev);
    if (n <= kSmallBatch) {
        if (shape.stream) run<kSmallBatch, true>(grads, n, shape.chunk_bytes, max_norm, norm, work, s);
        else run<kSmallBatch, false>(grads, n, shape.chunk_bytes, max_norm, norm, work, s);
    } else {
        if (shape.stream) run<kBatch, true>(grads, n, shape.chunk_bytes, max_norm, norm, work, s);
        else run<kBatch, false>(grads, n, shape.chunk_bytes, max_norm, norm, work, s);
    }
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
