// tiles.h -- which tile of a product a workgroup takes, on the device and the host
// alike.
#pragma once

#include <cstdint>

namespace wc {

constexpr uint32_t cdiv(uint64_t a, uint32_t b) { return (uint32_t)((a + b - 1) / b); }

constexpr uint32_t kDies = 8;
// The tile (m, n) of ms x ns that workgroup id takes, or none.  Workgroups go to the 8 dies in turn: each die gets a
// contiguous run of tiles (its L2 is its own), and within a run 4 tiles of m go with each tile of n, so that the tiles in
// work at one time share operands both ways.
constexpr bool tile_of(uint32_t id, uint32_t ms, uint32_t ns, uint32_t& m, uint32_t& n) {
    const uint32_t total = ms * ns, per = (total + kDies - 1) / kDies, t = id % kDies * per + id / kDies;
    if (id / kDies >= per || t >= total) return false;
    constexpr uint32_t kBand = 4;
    const uint32_t band = t / (kBand * ns), left = ms - band * kBand, width = left < kBand ? left : kBand;
    const uint32_t in = t - band * kBand * ns;
    m = band * kBand + in % width;
    n = in / width;
    return true;
}
constexpr uint32_t tile_grid(uint32_t ms, uint32_t ns) { return (ms * ns + kDies - 1) / kDies * kDies; }

}  // namespace wc
