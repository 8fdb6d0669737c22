// buffers.h -- buffer descriptors (gfx950): loads that check their range.
#pragma once

#include <cstdint>

namespace wc {

constexpr uint32_t kNoChunk = 0xFFFFFFF0u;      // a buffer offset beyond every operand: loads zeros
constexpr uint32_t kBufferWord = 0x00027000u;   // the last word of a descriptor of plain memory (no stride)

}  // namespace wc
