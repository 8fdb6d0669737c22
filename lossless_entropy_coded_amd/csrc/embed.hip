// embed.hip -- embedding lookup with scaling, from a bf16 table or from a
// 4-bit one with group scales, and the table's gradient.
//
//   out[t]     = scale * table[id[t]]            (rounded once to bf16)
//   dtable[v]  = scale * sum over t with id[t] = v of dout[t]
//
// An id outside [0, vocab) marks a token without a row (padding): its output
// row is zero and it gives no gradient.
//
// The lookup moves bytes only: a thread reads and writes 8 columns (16 bytes
// of bf16, 4 of codes), the tokens of a workgroup as many as fill it.
//
// The gradient sums each row's tokens in token order, so it is the same bits
// on every run.  Keys {id, token} are sorted: blocks of 4096 in LDS, then every
// key's place is its place in its block plus, for each other block, the number
// of smaller keys there (a binary search; keys are distinct).  The sorted
// tokens are cut into runs of kRun; a workgroup walks a run and sums each
// row's tokens in fp32.  A row whose tokens lie in one run is finished there;
// one that crosses runs leaves a partial sum per run, joined in run order by
// the last kernel.  Rows without tokens are written as zeros (unless the call
// accumulates) by further workgroups of the same launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/wc.h"

namespace wc {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
}

__device__ __forceinline__ int64_t id_at(const void* ids, uint32_t id_bytes, uint64_t t) {
    return id_bytes == 8 ? static_cast<const int64_t*>(ids)[t] : (int64_t) static_cast<const int32_t*>(ids)[t];
}

constexpr uint32_t kLookupThreads = 256;

struct LookupParams {
    const void* ids;
    uint16_t* out;
    const uint16_t* table;    // bf16 table
    const uint32_t* codes;    // 4-bit table
    const uint16_t* scales;
    const uint8_t* zeros;
    uint64_t n;
    uint32_t id_bytes, vocab, chunks;   // chunks: 8 columns each, per row
    uint32_t group, groups;
    uint32_t row_threads_log2;          // threads per token
    float scale;
};

template <bool kQ4>
__global__ __launch_bounds__(kLookupThreads) void embed_kernel(LookupParams p) {
    const uint32_t row_threads = 1u << p.row_threads_log2;
    const uint64_t t = (uint64_t)blockIdx.x * (kLookupThreads >> p.row_threads_log2) +
                       (threadIdx.x >> p.row_threads_log2);
    if (t >= p.n) return;
    const int64_t id = id_at(p.ids, p.id_bytes, t);
    const bool fits = id >= 0 && id < (int64_t)p.vocab;
    u32x4* const out = reinterpret_cast<u32x4*>(p.out) + t * p.chunks;
    for (uint32_t c = threadIdx.x & (row_threads - 1); c < p.chunks; c += row_threads) {
        u32x4 v = {0, 0, 0, 0};
        if (fits) {
            if (kQ4) {
                const uint32_t q = p.codes[(uint64_t)id * p.chunks + c];
                const uint64_t g = (uint64_t)id * p.groups + c * 8 / p.group;
                const float s = __uint_as_float((uint32_t)p.scales[g] << 16);
                const float z = p.zeros ? (float)p.zeros[g] : 8.0f;
                float f[8];
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) f[i] = s * ((float)((q >> (4 * i)) & 15u) - z) * p.scale;
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
            } else {
                v = reinterpret_cast<const u32x4*>(p.table)[(uint64_t)id * p.chunks + c];
                if (p.scale != 1.0f) {   // scale 1 keeps the words' bits, NaNs' too
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        v[i] = pack_bf16(bf16_lo(v[i]) * p.scale, bf16_hi(v[i]) * p.scale);
                }
            }
        }
        out[c] = v;
    }
}

// ---- gradient --------------------------------------------------------------

constexpr uint32_t kSortKeys = 4096;      // keys sorted in LDS by one workgroup
constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kRun = 32;             // sorted tokens per run
constexpr uint32_t kSumThreads = 256;
constexpr uint32_t kSumCols = kSumThreads * 8;   // columns per workgroup of the summing launch
constexpr uint32_t kFillRows = 16;        // rows per workgroup that looks for rows without tokens

struct GradParams {
    const uint16_t* dout;
    const void* ids;
    void* dtable;
    uint64_t* keys;       // blocks sorted (id << 32 | token)
    uint64_t* sorted;
    float* head;          // per run, the sum of its leading tokens whose row began in an earlier run
    float* tail;          // per run, the sum of its last row where that goes on in the next run
    uint32_t id_bytes, n, vocab, dim, runs;
    uint32_t bf16, accumulate;
    uint32_t col_blocks, row_blocks;
    float scale;
};

__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(GradParams p, uint64_t* out) {
    __shared__ uint64_t key[kSortKeys];
    const uint32_t base = blockIdx.x * kSortKeys;
    for (uint32_t i = threadIdx.x; i < kSortKeys; i += kSortThreads) {
        const uint32_t t = base + i;
        uint64_t k = ~0ull;
        if (t < p.n) {
            const int64_t id = id_at(p.ids, p.id_bytes, t);
            const uint32_t row = id >= 0 && id < (int64_t)p.vocab ? (uint32_t)id : p.vocab;
            k = (uint64_t)row << 32 | t;
        }
        key[i] = k;
    }
    __syncthreads();
    for (uint32_t size = 2; size <= kSortKeys; size <<= 1)
        for (uint32_t stride = size >> 1; stride > 0; stride >>= 1) {
            for (uint32_t i = threadIdx.x; i < kSortKeys / 2; i += kSortThreads) {
                const uint32_t a = 2 * i - (i & (stride - 1)), b = a + stride;
                const bool up = (a & size) == 0;
                const uint64_t x = key[a], y = key[b];
                if ((x > y) == up) key[a] = y, key[b] = x;
            }
            __syncthreads();
        }
    for (uint32_t i = threadIdx.x; i < kSortKeys && base + i < p.n; i += kSortThreads) out[base + i] = key[i];
}

__global__ __launch_bounds__(256) void embed_rank_kernel(GradParams p) {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= p.n) return;
    const uint64_t k = p.keys[i];
    const uint32_t mine = i / kSortKeys;
    uint32_t rank = i % kSortKeys;
    for (uint32_t base = 0, b = 0; base < p.n; base += kSortKeys, ++b) {
        if (b == mine) continue;
        uint32_t lo = 0, hi = min(kSortKeys, p.n - base);   // keys [0, lo) are smaller, [hi, ..) larger
        while (lo < hi) {
            const uint32_t mid = (lo + hi) / 2;
            if (p.keys[base + mid] < k) lo = mid + 1;
            else hi = mid;
        }
        rank += lo;
    }
    p.sorted[rank] = k;
}

__device__ __forceinline__ uint32_t row_of(uint64_t key) { return (uint32_t)(key >> 32); }

// dtable[row][col ..  col + 7] = scale * sum (+ what it held)
__device__ __forceinline__ void put_row(const GradParams& p, uint32_t row, uint32_t col, const float (&sum)[8]) {
    const uint64_t at = (uint64_t)row * p.dim + col;
    float v[8];
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) v[e] = p.scale * sum[e];
    if (p.bf16) {
        u32x4* const d = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.dtable) + at);
        u32x4 w;
        if (p.accumulate) {
            w = *d;
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) v[2 * e] += bf16_lo(w[e]), v[2 * e + 1] += bf16_hi(w[e]);
        }
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
        *d = w;
    } else {
        f32x4* const d = reinterpret_cast<f32x4*>(static_cast<float*>(p.dtable) + at);
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
            f32x4 w = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            if (p.accumulate) w += d[h];
            d[h] = w;
        }
    }
}

__device__ __forceinline__ void put_partial(float* part, uint64_t at, const float (&sum)[8]) {
    f32x4* const d = reinterpret_cast<f32x4*>(part + at);
    d[0] = f32x4{sum[0], sum[1], sum[2], sum[3]};
    d[1] = f32x4{sum[4], sum[5], sum[6], sum[7]};
}

__global__ __launch_bounds__(kSumThreads) void embed_sum_kernel(GradParams p) {
    const uint32_t cb = blockIdx.x % p.col_blocks, job = blockIdx.x / p.col_blocks;
    const uint32_t col = cb * kSumCols + threadIdx.x * 8;
    if (job >= p.runs) {   // rows without tokens
        __shared__ uint32_t empty[kFillRows];
        const uint32_t row0 = (job - p.runs) * kFillRows;
        if (threadIdx.x < kFillRows) {
            const uint32_t row = row0 + threadIdx.x;
            uint32_t lo = 0, hi = p.n;   // the first key of a row >= this one
            while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if (row_of(p.sorted[mid]) < row) lo = mid + 1;
                else hi = mid;
            }
            empty[threadIdx.x] = row < p.vocab && (lo == p.n || row_of(p.sorted[lo]) != row);
        }
        __syncthreads();
        if (col >= p.dim) return;
        for (uint32_t r = 0; r < kFillRows; ++r) {
            if (!empty[r]) continue;
            const uint64_t at = (uint64_t)(row0 + r) * p.dim + col;
            if (p.bf16) {
                *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.dtable) + at) = u32x4{0, 0, 0, 0};
            } else {
                f32x4* const d = reinterpret_cast<f32x4*>(static_cast<float*>(p.dtable) + at);
                d[0] = d[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
        return;
    }
    __shared__ uint64_t key[kRun + 2];   // the run's keys, the one before and the one after
    const uint32_t first = job * kRun, len = min(kRun, p.n - first);
    for (uint32_t i = threadIdx.x; i < len + 2; i += kSumThreads) {
        const uint32_t at = first + i;   // key[i] is sorted[first + i - 1]
        key[i] = at >= 1 && at <= p.n ? p.sorted[at - 1] : ~0ull;
    }
    __syncthreads();
    if (col >= p.dim) return;
    float sum[8] = {};
    for (uint32_t i = 0; i < len; ++i) {
        const uint32_t row = row_of(key[i + 1]);
        if (row >= p.vocab) return;   // tokens without a row come last
        const u32x4 w =
            *reinterpret_cast<const u32x4*>(p.dout + (uint64_t)(uint32_t)key[i + 1] * p.dim + col);
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) sum[2 * e] += bf16_lo(w[e]), sum[2 * e + 1] += bf16_hi(w[e]);
        const bool ends = first + i + 1 == p.n || row_of(key[i + 2]) != row;
        if (!ends && i + 1 < len) continue;
        const bool began_here = !(first > 0 && row_of(key[0]) == row);
        if (!began_here) put_partial(p.head, (uint64_t)job * p.dim + col, sum);
        else if (ends) put_row(p, row, col, sum);
        else put_partial(p.tail, (uint64_t)job * p.dim + col, sum);
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e) sum[e] = 0.0f;
    }
}

// A row that goes on from run to run: the partial of the run where it begins,
// then those of the runs after it, in order.
__global__ __launch_bounds__(kSumThreads) void embed_join_kernel(GradParams p) {
    const uint32_t cb = blockIdx.x % p.col_blocks, run = blockIdx.x / p.col_blocks;
    const uint32_t col = cb * kSumCols + threadIdx.x * 8;
    const uint32_t next = (run + 1) * kRun;
    const uint32_t row = row_of(p.sorted[next - 1]);
    if (row >= p.vocab || row_of(p.sorted[next]) != row) return;          // nothing goes on here
    const uint32_t first = run * kRun;
    if (first > 0 && row_of(p.sorted[first - 1]) == row && row_of(p.sorted[first]) == row) return;   // began earlier
    if (col >= p.dim) return;
    float sum[8];
    const f32x4* s = reinterpret_cast<const f32x4*>(p.tail + (uint64_t)run * p.dim + col);
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) sum[e] = s[e / 4][e % 4];
    for (uint32_t r = run + 1; r < p.runs && row_of(p.sorted[r * kRun]) == row; ++r) {
        s = reinterpret_cast<const f32x4*>(p.head + (uint64_t)r * p.dim + col);
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e) sum[e] += s[e / 4][e % 4];
    }
    put_row(p, row, col, sum);
}

constexpr uint64_t kAlign = 256;
uint64_t up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

struct GradLayout {
    uint64_t sorted, keys, head, tail, bytes;
    uint32_t runs;
};
GradLayout grad_layout(uint64_t n, uint32_t dim) {
    GradLayout l{};
    l.runs = (uint32_t)((n + kRun - 1) / kRun);
    l.sorted = 0;
    l.keys = up(n * 8, kAlign);
    l.head = l.keys + (n > kSortKeys ? up(n * 8, kAlign) : 0);
    l.tail = l.head + up((uint64_t)l.runs * dim * 4, kAlign);
    l.bytes = l.tail + up((uint64_t)l.runs * dim * 4, kAlign);
    return l;
}

bool ids_fit(const void* ids, uint32_t id_bytes) {
    return ids && (id_bytes == 4 || id_bytes == 8) && (reinterpret_cast<uintptr_t>(ids) & (id_bytes - 1)) == 0;
}
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int launch_lookup(LookupParams& p, bool q4, hipStream_t s) {
    p.row_threads_log2 = 0;
    while ((1u << p.row_threads_log2) < p.chunks && (1u << p.row_threads_log2) < kLookupThreads) ++p.row_threads_log2;
    const uint64_t per = kLookupThreads >> p.row_threads_log2, grid = (p.n + per - 1) / per;
    if (q4)
        hipLaunchKernelGGL(embed_kernel<true>, dim3((uint32_t)grid), dim3(kLookupThreads), 0, s, p);
    else
        hipLaunchKernelGGL(embed_kernel<false>, dim3((uint32_t)grid), dim3(kLookupThreads), 0, s, p);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}

}  // namespace
}  // namespace wc

using namespace wc;

extern "C" int wc_embed_async(const uint16_t* table, uint32_t vocab, uint32_t dim, const void* ids, uint32_t id_bytes,
                              uint64_t n, float scale, uint16_t* out, void* stream) {
    if (dim == 0 || dim % 8 != 0 || dim > WC_MAX_DIM || n > WC_MAX_TOKENS || vocab > WC_MAX_VOCAB)
        return WC_ERR_INVALID_ARG;
    if (n == 0) return WC_OK;
    if ((vocab != 0 && !aligned16(table)) || !aligned16(out) || !ids_fit(ids, id_bytes)) return WC_ERR_INVALID_ARG;
    LookupParams p{};
    p.ids = ids, p.id_bytes = id_bytes, p.n = n, p.out = out;
    p.table = table, p.vocab = vocab, p.chunks = dim / 8, p.scale = scale;
    return launch_lookup(p, false, static_cast<hipStream_t>(stream));
}

extern "C" int wc_embed_q4_async(const wc_q4_matrix* W, const void* ids, uint32_t id_bytes, uint64_t n, float scale,
                                 uint16_t* out, void* stream) {
    const int st = wc_q4_check(W);
    if (st != WC_OK) return st;
    if (n > WC_MAX_TOKENS) return WC_ERR_INVALID_ARG;
    if (n == 0) return WC_OK;
    if (!aligned16(out) || !ids_fit(ids, id_bytes)) return WC_ERR_INVALID_ARG;
    LookupParams p{};
    p.ids = ids, p.id_bytes = id_bytes, p.n = n, p.out = out;
    p.codes = reinterpret_cast<const uint32_t*>(W->codes), p.scales = W->scales, p.zeros = W->zeros;
    p.vocab = W->rows, p.chunks = W->cols / 8, p.scale = scale;
    p.group = W->group, p.groups = (W->cols + W->group - 1) / W->group;
    return launch_lookup(p, true, static_cast<hipStream_t>(stream));
}

extern "C" int wc_embed_grad_work_bytes(uint64_t n, uint32_t dim, uint64_t* work_bytes) {
    if (!work_bytes || dim == 0 || dim % 8 != 0 || dim > WC_MAX_DIM || n > WC_MAX_TOKENS)
        return WC_ERR_INVALID_ARG;
    *work_bytes = n ? grad_layout(n, dim).bytes : 0;
    return WC_OK;
}

extern "C" int wc_embed_grad_async(const uint16_t* dout, const void* ids, uint32_t id_bytes, uint64_t n, float scale,
                                   void* dtable, uint32_t out_kind, uint32_t vocab, uint32_t dim, int accumulate,
                                   void* work_dev, uint64_t work_bytes, void* stream) {
    if (dim == 0 || dim % 8 != 0 || dim > WC_MAX_DIM || n > WC_MAX_TOKENS || out_kind > WC_OUT_BF16 ||
        vocab > WC_MAX_VOCAB)
        return WC_ERR_INVALID_ARG;
    if (vocab == 0 || (n == 0 && accumulate)) return WC_OK;
    if (!aligned16(dtable)) return WC_ERR_INVALID_ARG;
    GradParams p{};
    const GradLayout l = grad_layout(n, dim);
    if (n) {
        if (!aligned16(dout) || !ids_fit(ids, id_bytes) || !work_dev ||
            (reinterpret_cast<uintptr_t>(work_dev) & (kAlign - 1)) || work_bytes < l.bytes)
            return WC_ERR_INVALID_ARG;
        uint8_t* const w = static_cast<uint8_t*>(work_dev);
        p.sorted = reinterpret_cast<uint64_t*>(w + l.sorted);
        p.keys = reinterpret_cast<uint64_t*>(w + l.keys);
        p.head = reinterpret_cast<float*>(w + l.head);
        p.tail = reinterpret_cast<float*>(w + l.tail);
    }
    p.dout = dout, p.ids = ids, p.id_bytes = id_bytes, p.dtable = dtable;
    p.n = (uint32_t)n, p.vocab = vocab, p.dim = dim, p.runs = l.runs;
    p.bf16 = out_kind == WC_OUT_BF16, p.accumulate = accumulate != 0, p.scale = scale;
    p.col_blocks = (dim + kSumCols - 1) / kSumCols;
    p.row_blocks = p.accumulate ? 0 : (vocab + kFillRows - 1) / kFillRows;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (n) {
        const bool one = n <= kSortKeys;
        hipLaunchKernelGGL(embed_sort_kernel, dim3((p.n + kSortKeys - 1) / kSortKeys), dim3(kSortThreads), 0, s, p,
                           one ? p.sorted : p.keys);
        if (!one) hipLaunchKernelGGL(embed_rank_kernel, dim3((p.n + 255) / 256), dim3(256), 0, s, p);
    }
    hipLaunchKernelGGL(embed_sum_kernel, dim3((p.runs + p.row_blocks) * p.col_blocks), dim3(kSumThreads), 0, s, p);
    if (p.runs > 1)
        hipLaunchKernelGGL(embed_join_kernel, dim3((p.runs - 1) * p.col_blocks), dim3(kSumThreads), 0, s, p);
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
