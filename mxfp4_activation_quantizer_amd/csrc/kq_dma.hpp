// Loads from memory straight into LDS for the MXFP4 products, and the order of
// the 16-byte chunks of a staged row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kq {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Chunk c (of eight) of staged row r is at slot c ^ swz8(r): a matrix read (32 rows of
// one chunk) then hits 32 distinct bank groups.
__device__ __forceinline__ int swz8(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Raw buffer descriptor in SGPRs: base, 32-bit record count (bytes); loads at
// or past the count return zero. What is compared with the count is the vector and the
// scalar offset together, by measurement on gfx950: 64 records read 16 dwords
// at scalar offset 0, 8 at 32 and none from 64 on, and 0 records none at any. The
// kernels keep the scalar offset at or below the count all the same, so that
// comparing the vector offset with the count less the scalar offset is no different.
__device__ __forceinline__ i32x4_t sdesc(const void *base, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4_t d;
    d.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    d.y = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu));
    d.z = __builtin_amdgcn_readfirstlane((int)bytes);
    d.w = 0x00020000;
    return d;
}

// 16 bytes per lane from the buffer straight into LDS: lane l's bytes land at
// lds + 16 l. M0 carries the LDS address and is restored afterwards; the
// compiler does not track these loads, so completion is waited for explicitly
// (vmcnt) before a barrier.
__device__ __forceinline__ void dma16(const i32x4_t &d, uint32_t lds, uint32_t voff, uint32_t soff) {
    uint32_t keep;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(keep)
        : "s"(lds), "v"(voff), "s"(d), "s"(soff)
        : "memory");
}

// 4 bytes per lane from the buffer straight into LDS: lane l's bytes land at lds + 4 l.
__device__ __forceinline__ void dma4(const i32x4_t &d, uint32_t lds, uint32_t voff) {
    uint32_t keep;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %2, %3, 0 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(keep)
        : "s"(lds), "v"(voff), "s"(d)
        : "memory");
}

}  // namespace kq
