// embed.hip -- embedding lookup with scaling, from a bf16 table or from a
// 4-bit one with group scales, and the table's gradient.
//
//   out[t]     = scale * table[id[t]]            (in fp32, rounded to bf16)
//   dtable[v]  = scale * sum over t with id[t] = v of dout[t]
//
// An id outside [0, vocab) marks a token without a row (padding): its output
// row is zero and it gives no gradient.
//
// The lookup moves bytes only: a thread reads and writes 8 columns (16 bytes
// of bf16, 4 of codes), the tokens of a workgroup as many as fill it.
//
// The gradient sums each row's tokens in a fixed order (token order within a
// run), so it is the same bits on every run.  Tokens are sorted by row: up to
// 8192 of them by counting for each the tokens before it, more in blocks of
// 4096 by a bitonic network whose keys (row, place in the block) fit 32 bits
// and stay in registers, four per lane, with all but the ten widest of its 78
// exchanges inside a wave (17 us; 38 with every exchange through LDS and 64-bit
// keys.  It is a chain of dependent steps: exchanges by lane swaps in place of
// __shfl_xor, and one v_med3 per key and step, take it to 16 to 19).  Then
// every token's place is its place in its block plus, for each other block, the
// number of smaller keys there: binary searches over the blocks' sorted rows,
// in LDS.  The sorted tokens are cut into runs of up to kRun; a workgroup walks a run, eight rows
// of the gradient on their way at a time, and sums each row's tokens in fp32.
// A row whose tokens lie in one run is finished there; one that crosses runs
// leaves a partial sum per run, joined in a fixed order by the last kernel.
// Rows without tokens are zero (unless the call accumulates): with a large table
// writing them is most of the bytes, and the memory's rate for writes bounds the
// call, so they are written beside the launches that leave the memory idle.
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

constexpr uint32_t kSortThreads = 1024;   // a workgroup sorts four keys per thread
constexpr uint32_t kRun = 32;             // sorted tokens per run at most
constexpr uint32_t kSumThreads = 256;
constexpr uint32_t kSumCols = kSumThreads * 8;   // columns per workgroup of the summing launch
constexpr uint32_t kAhead = 8;            // tokens of a run on their way at a time
constexpr uint32_t kFillRows = 16;        // rows per workgroup that looks for rows without tokens

struct GradParams {
    const uint16_t* dout;
    const void* ids;
    void* dtable;
    uint64_t* sorted;     // row << 32 | token, in order
    float* head;          // per run, the sum of its leading tokens whose row began in an earlier run
    float* tail;          // per run, the sum of its last row where that goes on in the next run
    uint32_t id_bytes, n, vocab, dim, runs, run_log2;
    uint32_t bf16, accumulate;
    uint32_t col_blocks, row_blocks;
    uint32_t filled;      // rows that are set to zero before this launch
    float scale;
};

struct SortParams {
    const void* ids;
    uint32_t id_bytes, n, vocab;
    uint32_t block_log2;   // keys per block: with a block's index beside it, a row fits 32 bits
    uint64_t* sorted;
    uint32_t* rows;        // per block, in order
    uint32_t* tokens;
    uint32_t blocks;
    uint32_t rank_blocks;  // workgroups that rank
    u32x4* fill;           // memory that further workgroups of the launch set to zero
    uint64_t fill_chunks;  // 16 bytes each
};

// The work of a filling workgroup, of the sorting launch's p.blocks and more: 16 bytes per thread, not kept in caches
// (with the whole table set here, 16384 tokens, 32768 x 4096, in a loop: 154 us; 32 bytes 160, 128: 168; kept: 172).
__device__ __forceinline__ void fill_zeros(const SortParams& p) {
    const uint64_t i = (uint64_t)(blockIdx.x - p.blocks) * blockDim.x + threadIdx.x;
    if (i < p.fill_chunks) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, p.fill + i);
}

__device__ __forceinline__ uint32_t row_at(const SortParams& p, uint32_t t) {
    const int64_t id = id_at(p.ids, p.id_bytes, t);
    return id >= 0 && id < (int64_t)p.vocab ? (uint32_t)id : p.vocab;
}

constexpr uint32_t kDirectTokens = 8192;
constexpr uint32_t kDirectThreads = 512;   // at most

// Few tokens: a token's place is the number of smaller keys (row, token), so
// each lane counts those of one token, a workgroup 64 tokens, each of its waves
// a part of the keys: 64 keys come into the lanes of a wave and go round as
// scalars, 3 operations per key and 64 tokens, which bound it: 4.2 us at 512
// tokens, 6.8 at 2048, 11 at 4096, 18 at 8192.  Against sorting and ranking, the
// whole gradient, us (5000 x 256 bf16): 512 tokens 13.5 and 15.7, 2048 17.1 and
// 20.1, 4096 20.4 and 26.4, 8192 29.6 and 35.4, 12000 37.2 and 38.0; 16384
// (32768 x 512) 49.9 and 45.1.
__global__ __launch_bounds__(kDirectThreads) void sort_direct_kernel(SortParams p) {
    if (blockIdx.x >= p.blocks) return fill_zeros(p);
    __shared__ uint32_t shared[kDirectThreads / 64][64];
    const uint32_t waves = blockDim.x >> 6;
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tile = blockIdx.x * 64, token = tile + lane;
    const uint32_t row = row_at(p, min(token, p.n - 1));
    const uint32_t per = ((p.n + 63) / 64 + waves - 1) / waves * 64;
    const uint32_t begin = min(wave * per, p.n), end = min(begin + per, p.n);
    uint32_t place = 0;
    uint32_t next = begin + lane < end ? row_at(p, begin + lane) : ~0u;   // (smaller than no key)
    for (uint32_t from = begin; from < end; from += 64) {
        const uint32_t keys = next;
        next = from + 64 + lane < end ? row_at(p, from + 64 + lane) : ~0u;
        if (from != tile) {
            const uint32_t less = row + (from < tile);   // earlier tokens of the same row come before
#pragma unroll
            for (uint32_t k = 0; k < 64; ++k) place += (uint32_t)__builtin_amdgcn_readlane((int)keys, k) < less;
        } else {
#pragma unroll
            for (uint32_t k = 0; k < 64; ++k)
                place += (uint32_t)__builtin_amdgcn_readlane((int)keys, k) < row + (k < lane);
        }
    }
    shared[wave][lane] = place;
    __syncthreads();
    if (wave != 0 || token >= p.n) return;
    for (uint32_t w = 1; w < waves; ++w) place += shared[w][lane];
    p.sorted[place] = (uint64_t)row << 32 | token;
}

// The keys of a block in order: four per thread, keys 4 t .. 4 t + 3.
__global__ __launch_bounds__(kSortThreads) void sort_block_kernel(SortParams p) {
    __shared__ u32x4 shared[kSortThreads];
    if (blockIdx.x >= p.blocks) return fill_zeros(p);
    const uint32_t tid = threadIdx.x, base = blockIdx.x << p.block_log2;
    const uint32_t count = min(p.n - base, 1u << p.block_log2);
    u32x4 key;
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t i = tid * 4 + e;
        uint32_t k = ~0u;
        if (i < count) k = row_at(p, base + i) << p.block_log2 | i;
        key[e] = k;
    }
    const auto order = [&](uint32_t a, uint32_t b, bool up) {   // key[a] before key[b], or after it
        const uint32_t lo = min(key[a], key[b]), hi = max(key[a], key[b]);
        key[a] = up ? lo : hi;
        key[b] = up ? hi : lo;
    };
    order(0, 1, true);
    order(2, 3, false);
    for (uint32_t size = 4; size <= 1u << p.block_log2; size <<= 1) {
        const bool up = (tid * 4 & size) == 0;
        for (uint32_t stride = size >> 1; stride >= 4; stride >>= 1) {
            const uint32_t far = stride / 4;
            u32x4 other;
            if (far >= 64) {
                __syncthreads();
                shared[tid] = key;
                __syncthreads();
                other = shared[tid ^ far];
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) other[e] = (uint32_t)__shfl_xor((int)key[e], (int)far);
            }
            const bool low = ((tid & far) == 0) == up;
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) key[e] = low ? min(key[e], other[e]) : max(key[e], other[e]);
        }
        order(0, 2, up);
        order(1, 3, up);
        order(0, 1, up);
        order(2, 3, up);
    }
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
        const uint32_t i = tid * 4 + e;
        if (i >= count) continue;
        const uint32_t row = key[e] >> p.block_log2, token = base + (key[e] & ((1u << p.block_log2) - 1));
        p.rows[base + i] = row;
        p.tokens[base + i] = token;
    }
}

constexpr uint32_t kRankThreads = 1024;
constexpr uint32_t kRankKeys = 32768;   // rows of other blocks in LDS at a time (128 KB)
constexpr uint32_t kRankFillers = 240;  // filling workgroups at most: about one per CU, as the LDS allows (480 are no faster)

// Every token's place: its place in its block, and the smaller keys of the
// other blocks, whose sorted rows come through LDS.
__global__ __launch_bounds__(kRankThreads) void sort_rank_kernel(SortParams p) {
    if (blockIdx.x >= p.rank_blocks) {
        const uint64_t step = (uint64_t)(gridDim.x - p.rank_blocks) * kRankThreads;
        for (uint64_t at = (uint64_t)(blockIdx.x - p.rank_blocks) * kRankThreads + threadIdx.x; at < p.fill_chunks; at += step)
            __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, p.fill + at);
        return;
    }
    __shared__ uint32_t rows[kRankKeys];
    const uint32_t i = blockIdx.x * kRankThreads + threadIdx.x, log2 = p.block_log2, block = 1u << log2;
    const bool there = i < p.n;
    const uint32_t row = there ? p.rows[i] : 0, mine = i >> log2;
    uint32_t rank = i & (block - 1);
    for (uint32_t from = 0; from < p.n; from += kRankKeys) {
        __syncthreads();
        for (uint32_t k = threadIdx.x; k < kRankKeys; k += kRankThreads)
            rows[k] = from + k < p.n ? p.rows[from + k] : ~0u;   // sorted last in its block
        __syncthreads();
        for (uint32_t b = 0; b < kRankKeys >> log2 && from + (b << log2) < p.n; ++b) {
            const uint32_t at = (from >> log2) + b;
            if (at == mine) continue;
            // earlier blocks' keys of the same row or a smaller one, later blocks' of a smaller one
            const uint32_t less = row + (at < mine);
            const uint32_t* const in = rows + (b << log2);
            uint32_t before = 0;
            for (uint32_t step = block; step > 0; step >>= 1)
                if (before + step <= block && in[before + step - 1] < less) before += step;
            rank += before;
        }
    }
    if (there) p.sorted[rank] = (uint64_t)row << 32 | p.tokens[i];
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
        const uint32_t row0 = p.filled + (job - p.runs) * kFillRows;
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
        // 16 bytes per lane and store, side by side: whole lines, not kept in caches
        const uint32_t row_chunks = p.dim / 8 << !p.bf16, chunk0 = cb * kSumThreads << !p.bf16;
        const uint32_t end = min(row_chunks, chunk0 + (kSumThreads << !p.bf16));
        for (uint32_t r = 0; r < kFillRows; ++r) {
            if (!empty[r]) continue;
            u32x4* const row = static_cast<u32x4*>(p.dtable) + (uint64_t)(row0 + r) * row_chunks;
            for (uint32_t c = chunk0 + threadIdx.x; c < end; c += kSumThreads)
                __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, row + c);
        }
        return;
    }
    __shared__ uint64_t key[kRun + 2];   // the run's keys, the one before and the one after
    const uint32_t first = job << p.run_log2, len = min(1u << p.run_log2, p.n - first);
    for (uint32_t i = threadIdx.x; i < len + 2; i += kSumThreads) {
        const uint32_t at = first + i;   // key[i] is sorted[first + i - 1]
        key[i] = at >= 1 && at <= p.n ? p.sorted[at - 1] : ~0ull;
    }
    __syncthreads();
    if (col >= p.dim) return;
    float sum[8] = {};
    for (uint32_t i0 = 0; i0 < len; i0 += kAhead) {
        u32x4 w[kAhead];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint64_t at = key[min(i0 + k, len - 1) + 1];   // past the run: its last token again, unused
            w[k] = *reinterpret_cast<const u32x4*>(p.dout + (uint64_t)(uint32_t)at * p.dim + col);
        }
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t i = i0 + k;
            if (i >= len) return;
            const uint32_t row = row_of(key[i + 1]);
            if (row >= p.vocab) return;   // tokens without a row come last
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) sum[2 * e] += bf16_lo(w[k][e]), sum[2 * e + 1] += bf16_hi(w[k][e]);
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
}

constexpr uint32_t kJoinSlices = 8;                              // of a row's runs
constexpr uint32_t kJoinCols = kSumThreads / kJoinSlices * 8;    // columns of a workgroup at a time
constexpr uint32_t kJoinBlocks = 4;                              // workgroups per run at most

// A row that goes on from run to run: the partial of the run where it begins
// and those of the runs after it, in order within each of 8 slices of them,
// then the slices in order.
__global__ __launch_bounds__(kSumThreads) void embed_join_kernel(GradParams p, uint32_t join_blocks) {
    const uint32_t run = blockIdx.x / join_blocks;
    const uint32_t first = run << p.run_log2, next = first + (1u << p.run_log2);
    // most runs have none, and are done after one trip to memory
    const uint32_t row = row_of(p.sorted[next - 1]), after = row_of(p.sorted[next]);
    const uint32_t before = row_of(p.sorted[first > 0 ? first - 1 : 0]);
    if (row >= p.vocab || after != row || (first > 0 && before == row)) return;
    // the runs that the row goes on in: up to the one that holds its last token, looked for in growing steps
    uint32_t lo = next + 1, step = 1u << p.run_log2;   // tokens up to lo - 1 are the row's
    while (lo + step <= p.n && row_of(p.sorted[lo + step - 1]) == row) lo += step, step *= 2;
    for (; step > 0; step >>= 1)
        if (lo + step <= p.n && row_of(p.sorted[lo + step - 1]) == row) lo += step;
    const uint32_t runs = ((lo - 1) >> p.run_log2) - run, per = (runs + kJoinSlices - 1) / kJoinSlices;
    const uint32_t slice = threadIdx.x / (kSumThreads / kJoinSlices), lane = threadIdx.x % (kSumThreads / kJoinSlices);
    const uint32_t begin = run + 1 + slice * per, end = min(begin + per, run + 1 + runs);
    __shared__ f32x4 shared[2][kSumThreads];
    for (uint32_t col0 = blockIdx.x % join_blocks * kJoinCols; col0 < p.dim; col0 += join_blocks * kJoinCols) {
        const uint32_t col = col0 + lane * 8;
        const bool inside = col < p.dim;
        float sum[8] = {};
        if (inside) {
            if (slice == 0) {
                const f32x4* const tail = reinterpret_cast<const f32x4*>(p.tail + (uint64_t)run * p.dim + col);
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e) sum[e] = tail[e / 4][e % 4];
            }
            for (uint32_t r0 = begin; r0 < end; r0 += kAhead) {
                f32x4 part[kAhead][2];
#pragma unroll
                for (uint32_t k = 0; k < kAhead; ++k) {
                    const f32x4* const from =
                        reinterpret_cast<const f32x4*>(p.head + (uint64_t)min(r0 + k, end - 1) * p.dim + col);
                    part[k][0] = from[0], part[k][1] = from[1];
                }
#pragma unroll
                for (uint32_t k = 0; k < kAhead; ++k)
                    if (r0 + k < end)
#pragma unroll
                        for (uint32_t e = 0; e < 8; ++e) sum[e] += part[k][e / 4][e % 4];
            }
        }
        __syncthreads();
        shared[0][threadIdx.x] = f32x4{sum[0], sum[1], sum[2], sum[3]};
        shared[1][threadIdx.x] = f32x4{sum[4], sum[5], sum[6], sum[7]};
        __syncthreads();
        if (slice != 0 || !inside) continue;
#pragma unroll
        for (uint32_t k = 1; k < kJoinSlices; ++k)
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) sum[e] += shared[e / 4][threadIdx.x + k * (kSumThreads / kJoinSlices)][e % 4];
        put_row(p, row, col, sum);
    }
}

constexpr uint64_t kAlign = 256;
uint64_t up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

struct GradLayout {
    uint64_t sorted, scratch, head, tail, bytes;
    uint32_t runs, run_log2;
};
// Runs of 32 tokens, or of 16 or 8 where that leaves fewer than 1024
// workgroups: eight tokens are on their way at a time, so longer runs of a
// small batch only wait.
GradLayout grad_layout(uint64_t n, uint32_t dim) {
    GradLayout l{};
    l.run_log2 = 5;
    static_assert(kRun == 1u << 5, "the longest run");
    while (l.run_log2 > 3 && (n >> l.run_log2) * ((dim + kSumCols - 1) / kSumCols) < 1024) --l.run_log2;
    l.runs = (uint32_t)((n + (1u << l.run_log2) - 1) >> l.run_log2);
    l.sorted = 0;
    l.scratch = up(n * 8, kAlign);
    l.head = l.scratch + up(n * 8, kAlign);
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

// Tokens sorted by id, then by token: sorted[i] = row << 32 | token, row = vocab
// for ids (id_bytes 4 or 8 each) outside [0, vocab).  scratch: 2 n words.  1 <=
// n <= 2^20, vocab <= 2^22.  One launch up to 8192 tokens, else two.  The first
// one also sets fill_bytes at `fill` to zero, the second one more_bytes behind
// them (multiples of 16; 0 if there is one launch).
void launch_sort_ids(const void* ids, uint32_t id_bytes, uint32_t n, uint32_t vocab, uint64_t* sorted,
                     uint32_t* scratch, hipStream_t stream, void* fill, uint64_t fill_bytes, uint64_t more_bytes) {
    SortParams p{};
    p.ids = ids, p.id_bytes = id_bytes, p.n = n, p.vocab = vocab, p.sorted = sorted;
    p.fill = static_cast<u32x4*>(fill), p.fill_chunks = fill_bytes / 16;
    const auto blocks = [&](uint32_t threads) {   // of the first launch, those that fill among them
        return dim3((uint32_t)(p.blocks + (p.fill_chunks + threads - 1) / threads));
    };
    if (n <= kDirectTokens) {
        p.blocks = (n + 63) / 64;
        const uint32_t threads = n <= 1024 ? kDirectThreads / 2 : kDirectThreads;   // small workgroups fill faster
        hipLaunchKernelGGL(sort_direct_kernel, blocks(threads), dim3(threads), 0, stream, p);
        return;
    }
    p.block_log2 = 12;
    while (((uint64_t)(vocab + 1) << p.block_log2) > 0x100000000ull) --p.block_log2;
    const uint32_t block = 1u << p.block_log2;
    p.blocks = (n + block - 1) / block;
    p.rows = scratch, p.tokens = scratch + n;
    hipLaunchKernelGGL(sort_block_kernel, blocks(block / 4), dim3(block / 4), 0, stream, p);
    p.rank_blocks = (n + kRankThreads - 1) / kRankThreads;
    p.fill += p.fill_chunks, p.fill_chunks = more_bytes / 16;
    const uint64_t groups = (p.fill_chunks + kRankThreads - 1) / kRankThreads;
    hipLaunchKernelGGL(sort_rank_kernel, dim3(p.rank_blocks + (uint32_t)(groups < kRankFillers ? groups : kRankFillers)),
                       dim3(kRankThreads), 0, stream, p);
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
    p.group = W->group, p.groups = W->group < W->cols ? (W->cols + W->group - 1) / W->group : 1;
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
    uint32_t* scratch = nullptr;
    const GradLayout l = grad_layout(n, dim);
    if (n) {
        if (!aligned16(dout) || !ids_fit(ids, id_bytes) || !work_dev ||
            (reinterpret_cast<uintptr_t>(work_dev) & (kAlign - 1)) || work_bytes < l.bytes)
            return WC_ERR_INVALID_ARG;
        uint8_t* const w = static_cast<uint8_t*>(work_dev);
        p.sorted = reinterpret_cast<uint64_t*>(w + l.sorted);
        scratch = reinterpret_cast<uint32_t*>(w + l.scratch);
        p.head = reinterpret_cast<float*>(w + l.head);
        p.tail = reinterpret_cast<float*>(w + l.tail);
    }
    p.dout = dout, p.ids = ids, p.id_bytes = id_bytes, p.dtable = dtable;
    p.n = (uint32_t)n, p.vocab = vocab, p.dim = dim, p.runs = l.runs, p.run_log2 = l.run_log2;
    p.bf16 = out_kind == WC_OUT_BF16, p.accumulate = accumulate != 0, p.scale = scale;
    p.col_blocks = (dim + kSumCols - 1) / kSumCols;
    // Rows without tokens.  What the sort's few workgroups leave idle sets the table's first rows to zero, those with
    // tokens too, which are written again: as many bytes as take about as long as the sorting launch, and the ranking
    // one.  The others are written by the summing launch, whose reads leave some of the memory idle, row by row where
    // there are no tokens; few tokens have no ranking and a short summing launch, so there all rows are set beside the
    // sort.  Measured on inputs that rotate past the caches, us (nothing ahead; 128 MiB beside the sort; that and 6 KiB
    // per token beside the ranking, as here; the same, and the rest beside the sort; one set of inputs in a loop, whose
    // gradients stay in the cache, takes up to 11 us less; a table of its own for each call too, up to 14 more):
    //   32768 x 4096 fp32, 16384 tokens    160  149  140  160
    //   131072 x 512 fp32, 16384 tokens     84   69   61   76
    //   131072 x 4096 bf16, 65536 tokens   390  380  352  371
    //   32000 x 4096 bf16, 32768 tokens    155  144  136  149
    //   32768 x 4096 fp32, 8192 tokens     140  125    -  120
    //   32000 x 4096 fp32, 2048 tokens     118  111    -  102
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint64_t sort_bytes = 0, rank_bytes = 0;
    if (n && !p.accumulate) {
        const uint64_t row_bytes = (uint64_t)dim * (p.bf16 ? 2 : 4);
        const bool one = n <= kDirectTokens;
        const uint64_t first = one ? 32ull << 30 : 128ull << 20;   // (a launch holds fewer than 2^32 threads of 16 bytes)
        const uint64_t second = one ? 0 : n * 6144;
        const uint64_t rows = (first + second) / row_bytes;
        p.filled = rows < vocab ? (uint32_t)rows : vocab;
        const uint64_t bytes = p.filled * row_bytes;
        sort_bytes = bytes < first ? bytes : first;
        rank_bytes = bytes - sort_bytes;
    }
    p.row_blocks = p.accumulate ? 0 : (vocab - p.filled + kFillRows - 1) / kFillRows;
    if (n) launch_sort_ids(ids, id_bytes, p.n, vocab, p.sorted, scratch, s, dtable, sort_bytes, rank_bytes);
    hipLaunchKernelGGL(embed_sum_kernel, dim3((p.runs + p.row_blocks) * p.col_blocks), dim3(kSumThreads), 0, s, p);
    if (p.runs > 1) {
        const uint32_t blocks = (dim + kJoinCols - 1) / kJoinCols, join_blocks = blocks < kJoinBlocks ? blocks : kJoinBlocks;
        hipLaunchKernelGGL(embed_join_kernel, dim3((p.runs - 1) * join_blocks), dim3(kSumThreads), 0, s, p, join_blocks);
    }
    return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP;
}
