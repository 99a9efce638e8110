// lds_dma.h -- direct global -> LDS loads of the LDS-staged matrix-core loops.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Direct global -> LDS loads (16 or 4 bytes per lane; lane l's bytes land
// at lds + 16 l, or 4 l).  Written as inline asm so that the compiler does
// not treat every later LDS read as depending on them (it would wait for all
// of them, a full drain, before each read); the main loop waits for them
// itself.  M0 (the LDS base) is saved and restored inside the block.
typedef __attribute__((address_space(3))) const void lds_cvoid_t;
__device__ inline uint32_t lds_addr(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_cvoid_t*)p);
}
__device__ inline void dma16(const uint8_t* src, uint32_t lds) {
    uint32_t save;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(save)
        : "v"(src), "s"(lds)
        : "memory");
}
__device__ inline void dma4(const uint8_t* src, uint32_t lds) {
    uint32_t save;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(save)
        : "v"(src), "s"(lds)
        : "memory");
}

// The same with a scalar base address and a 32-bit offset per lane.  No
// memory clobber: the loop's own wait and barrier orders them, and the
// compiler may keep them among its other work.
__device__ inline void dma16s(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t save;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %2\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(save)
        : "v"(off), "s"(base), "s"(lds));
}
__device__ inline void dma4s(const uint8_t* base, uint32_t off, uint32_t lds) {
    uint32_t save;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %1, %2\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(save)
        : "v"(off), "s"(base), "s"(lds));
}

}  // namespace moe
