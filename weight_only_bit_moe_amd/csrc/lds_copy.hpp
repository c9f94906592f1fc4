// Direct copies from memory into LDS, and the places of operand rows there,
// shared by the 8-bit products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "window.hpp"

namespace wna16 {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

template <class T> struct __attribute__((packed, aligned(sizeof(T)))) Out4 { T v[4]; };

// LDS byte address of a __shared__ pointer.
__device__ __forceinline__ uint32_t lds_of(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)(p);
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Lane l's 16 bytes at base + voff land at LDS address lds + l * 16.  base and
// lds are wave-uniform.  Inline asm, so that the compiler does not make every
// later LDS read wait for all copies in flight; the caller waits with vmcnt.
__device__ __forceinline__ void copy16_to_lds(const void *base_in, uint32_t voff, uint32_t lds_in)
{
    const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_in);
    const uint64_t b = reinterpret_cast<uintptr_t>(base_in);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    const void *base = reinterpret_cast<const void *>(((uint64_t)hi << 32) | (uint64_t)lo);
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base),
                 "s"(lds)
                 : "memory", "m0");
}

// The same from a buffer: voff of the lane and soff of the wave are added.  A piece at or
// past the buffer's end by voff alone is not read; whether soff counts there too is not
// relied on, so a piece inside by voff has to be inside with soff as well (window_of).
__device__ __forceinline__ void copy16_to_lds(v4i buffer, uint32_t voff, uint32_t soff_in,
                                              uint32_t lds_in)
{
    const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_in);
    const uint32_t soff = (uint32_t)__builtin_amdgcn_readfirstlane((int)soff_in);
    asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff),
                 "s"(buffer), "s"(soff), "s"(lds)
                 : "memory", "m0");
}
// Each active lane l's 4 bytes at voff land at lds + l * 4.
__device__ __forceinline__ void copy4_to_lds(v4i buffer, uint32_t voff, uint32_t lds_in)
{
    const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_in);
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff),
                 "s"(buffer), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Descriptor of `bytes` bytes at a wave-uniform address: raw, 32-bit elements.
__device__ __forceinline__ v4i buffer_of(const void *p, uint32_t bytes)
{
    const uint64_t b = reinterpret_cast<uintptr_t>(p);
    return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               __builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xffffu)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Place of a row's 16-byte piece c among the 8 of its 128-byte LDS row: the 16
// rows that one MFMA operand read touches are spread over all banks.
__device__ __forceinline__ int place(int row, int c) { return c ^ ((row >> 1) & 7); }

template <int N>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace

}  // namespace wna16
