// gemm_fp8_plan.h -- which kernel a product with e4m3 matrices takes: its tile, its
// splits of the columns, and its variant, by the sizes and the type of the results
// alone.  Host code, without the runtime's headers.
#pragma once

#include <cstdint>

#include "../../include/wc.h"
#include "tiles.h"

namespace wc {

// Elements of one split's sums: they begin on 16 bytes.
constexpr uint64_t split_elems(uint64_t tokens, uint32_t rows) { return (tokens * rows + 3) / 4 * 4; }

constexpr uint32_t kCus = 256;
constexpr uint32_t kFewTokens = 32;

// Tiles and splits of more tokens are those that a model of the time likes best.  It knows what a tile takes per block of
// columns, which is fitted to the times below: 36 to 41 bytes per ns and CU from 32 x 32 to 256 x 256, or, where codes are
// made bf16, down to half of that.  (No unit is at its limit there: of 256 tokens x 28672 x 8192 the matrix cores are busy
// 26% of the time and memory gives 3.0 TB/s.  A tile's copies, reads from LDS and products wait for one another: 94 us, of
// columns that stay in L2 74, without copies 62.)  It adds a workgroup's start and end, 3 us, and for joining splits a launch
// of 2.5 us and their sums, written and read at 4 TB/s.  Few and small tiles leave CUs idle, large ones re-read the least.
// Measured (us, tile:splits; * what the model takes):
//                                32x32   32x64   64x64     128x64    128x128   256x128   256x256
//    64 tokens x 4096 x 4096       7.6*   12.7    12.8       -         -         -         -
//   128 x 4096 x 4096             13.1     9.3*   10.8      14.2:2     -         -         -
//   256 x 4096 x 4096              -      16.4    11.3*     15.2      17.7:4     -         -
//    64 x 28672 x 8192             -       -      61.2      49.1*     49.7      63.5:2     -
//   128 x 4096 x 14336             -       -       -        28.3:4    28.7:8*   29.0:16    -
//   128 x 8192 x 28672             -       -       -        86.3:2    69.4:4*   61.9:8     -     (the model is wrong here)
//   128 x 28672 x 8192             -       -       -        82.2      62.3*     69.1:2     -
//   512 x 4096 x 4096              -       -      20.0      16.4*     22.0       -         -
//   512 x 14336 x 4096             -       -      94.2      62.6      57.5      45.9*     58.9
//  1000 x 8192 x 8192              -       -       -         122       101      82.6*      105
//  1024 x 14336 x 4096             -       -       -         110       103      78.9      63.8*
//  5000 x 300 x 9008 fp32          -       -       -        52.0*     52.8:4    72.5:2
//   512 x 14336 x 4096 fp32        -       161     104      82.1      70.9      65.2*
//  1024 x 4096 x 4096 fp32         -       -      56.9      45.0*     54.9      48.3:2
struct Kind {
    uint32_t bm, bn, per_cu;   // workgroups per CU (LDS)
    double us;                 // per block of columns
};
constexpr uint32_t kKinds = 7, kBig = kKinds - 1;   // the last of codes alone, and without splits
constexpr uint32_t kHalf = 3, kSquare = 4;           // 128 x 64 and 128 x 128
constexpr Kind kCodeKinds[kKinds] = {{32, 32, 1, 0.2}, {32, 64, 1, 0.3}, {64, 64, 1, 0.4}, {128, 64, 2, 0.6},
                                     {128, 128, 1, 0.8}, {256, 128, 1, 1.4}, {256, 256, 1, 1.6}};
constexpr Kind kExactKinds[kBig] = {{32, 32, 1, 0.26}, {32, 64, 1, 0.4}, {64, 64, 1, 0.42}, {128, 64, 2, 0.65},
                                    {128, 128, 2, 1.35}, {256, 128, 1, 2.0}};

// Groups of few tokens: of 16, 32 and 64 rows, and, of 17 to 32 tokens, of 16 and 32.
enum FewKind : uint32_t { kFew16, kFew32, kFew64, kFewPairs16, kFewPairs32, kFewKinds };

// Rows of a group of few tokens, and its waves and stages (us): past 4096 rows there are groups enough of 32 rows, which
// share the work on the tokens; from 10240 to 16384 rows groups of 64, one per CU, are all in work at once.
//                          16 rows, 8 waves   32 rows, 4 waves   64 rows, 4 waves
//    1 token  x 1024 x 4096        4.8               5.9                8.4
//    8 tokens x 4096 x 14336      12.3              16.0               24.8
//    1 x 4608 x 8192              12.1               9.4               14.3
//   16 x 10240 x 8192             20.4              21.0               17.9
//   16 x 14336 x 4096             15.9              13.2               12.3
//   16 x 16384 x 8192             29.7              24.4               23.6
//   16 x 24576 x 8192             44.9              36.3               42.4
//   16 x 57344 x 8192             98.3              80.8               85.4
// 17 to 32 tokens: 16 and 32 rows, 4 waves of 2 stages: 24 x 1024 x 4096 6.6 and 8.0, 32 x 4096 x 14336 19.2 and 24.5, 32 x
// 5120 x 8192 19.6 and 14.7, 32 x 28672 x 8192 69 and 52.
constexpr uint32_t kNarrowRows = 4096, kTallFrom = 10240, kTallRows = 16384;
constexpr FewKind few_kind(uint32_t rows, uint64_t tokens) {
    if (tokens > 16) return rows <= kNarrowRows ? kFewPairs16 : kFewPairs32;
    if (rows <= kNarrowRows) return kFew16;
    return rows >= kTallFrom && rows <= kTallRows ? kFew64 : kFew32;
}

struct GemmPlan {
    bool few;                        // kind: a FewKind, else a tile's
    uint32_t kind, splits, split_blocks;
    bool once;                       // the matrix is read once, past the caches
    bool pair;                       // of 128 x 64: two groups of waves
    uint64_t work_bytes;
};

// A matrix that one tile of tokens takes whole is read once, and past the caches (us, and through them): 64 tokens x 28672 x
// 8192 52.7 and 59.2, 128 tokens 62.9 and 68.7, 64 tokens x 14336 x 4096 17.9 and 19.6; not if two do: 128 tokens x 4096 x
// 14336 in tiles of 64, 28.3 and 26.3.
// (An fp32 tile of 128 x 128 is never the best one where it takes all tokens: of more than 256 such tiles 256 x 128 costs
// less, of fewer 128 x 64.)
constexpr bool reads_once(uint32_t kind, bool exact, uint64_t tokens) {
    const uint32_t bn = exact ? kExactKinds[kind].bn : kCodeKinds[kind].bn;
    return bn > kFewTokens && tokens <= bn && kind != kBig && !(exact && kind == kSquare);
}

inline GemmPlan plan_of(uint32_t rows, uint32_t cols, uint64_t tokens, bool exact) {
    const uint32_t blocks = cdiv(cols, WC_FP8_BLOCK);
    if (tokens <= kFewTokens) return {true, few_kind(rows, tokens), 1, blocks, false, false, 0};
    GemmPlan best{};
    double best_us = 1e300;
    for (uint32_t k = 0; k < (exact ? kBig : kKinds); ++k) {
        const Kind& kind = exact ? kExactKinds[k] : kCodeKinds[k];
        const uint64_t tiles = (uint64_t)cdiv(rows, kind.bm) * cdiv(tokens, kind.bn);
        for (uint32_t s = 1; s <= 16; s *= 2) {
            if (s > 1 && (k == kBig || blocks < 8 * s || tiles * s > kCus * kind.per_cu)) break;
            const uint32_t per = cdiv(blocks, s);
            const uint64_t groups = tiles * s;
            const double us = 3.0 * (double)((groups + kCus * kind.per_cu - 1) / (kCus * kind.per_cu)) +
                              (double)((groups + kCus - 1) / kCus) * per * kind.us +
                              (s > 1 ? 2.5 + (double)s * (double)tokens * rows * 8 / 4e6 : 0.0);
            if (us < best_us) best_us = us, best.kind = k, best.splits = cdiv(blocks, per), best.split_blocks = per;
        }
    }
    best.once = reads_once(best.kind, exact, tokens);
    // where no CU has two workgroups, so that as much is on its way (64 tokens x 28672 x 8192, us: 48.7, and 56.3 with one)
    best.pair = best.kind == kHalf && cdiv(rows, 128) * (uint64_t)cdiv(tokens, 64) * best.splits <= kCus;
    best.work_bytes = best.splits > 1 ? best.splits * split_elems(tokens, rows) * 4 : 0;
    return best;
}

}  // namespace wc
