// lds_copy.h -- copies from memory straight into LDS (gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "buffers.h"

namespace wc {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The byte offset in LDS of a pointer into it.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// A buffer of `bytes` bytes at p: accesses beyond it load zeros.
__device__ __forceinline__ u32x4 buffer_words(const void* p, uint32_t bytes) {
    const uint64_t addr = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)addr, (uint32_t)(addr >> 32) & 0xFFFFu, bytes, kBufferWord};
}

// Start copying 16 bytes per lane from a buffer to consecutive LDS places from
// `to` (uniform over the wave).  It writes no register and is counted by vmcnt,
// in order with other loads; the caller does the waiting that is needed before
// LDS is read.  In assembly because the compiler, for the builtin, waits for
// every such copy before each transposing LDS read; but then it does not count
// the copy when it waits for other loads, so a kernel keeps no loads into
// registers on their way beside it.  Nor does it add the wait state that a
// memory instruction with LDS needs behind a write of m0: the s_nop is that one
// (without it the copy may go to the place of the copy before).
__device__ __forceinline__ void copy_to_lds(uint32_t to, const u32x4& rsrc, uint32_t offset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(offset),
                 "s"(rsrc)
                 : "memory", "m0");
}

// The same from offset + uniform (uniform over the wave, at most the buffer's size).
__device__ __forceinline__ void copy_to_lds(uint32_t to, const u32x4& rsrc, uint32_t offset, uint32_t uniform) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(offset),
                 "s"(rsrc), "s"(uniform)
                 : "memory", "m0");
}

// The same past the caches, for what is read once.
__device__ __forceinline__ void copy_once_to_lds(uint32_t to, const u32x4& rsrc, uint32_t offset, uint32_t uniform) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(to), "v"(offset),
                 "s"(rsrc), "s"(uniform)
                 : "memory", "m0");
}

// The same with 4 bytes per lane.
__device__ __forceinline__ void copy_words_to_lds(uint32_t to, const u32x4& rsrc, uint32_t offset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(offset),
                 "s"(rsrc)
                 : "memory", "m0");
}

}  // namespace wc
