// lds_dma.hpp - buffer resources and direct buffer->LDS loads of gfx950 for the
// grouped GEMMs.
#pragma once

#include "common.hpp"

namespace cmoe {

typedef int32_t Rsrc __attribute__((ext_vector_type(4)));

// Resource of a raw byte buffer: base address, size in bytes (loads past it give
// zeros instead of touching memory), stride 0.
__device__ __forceinline__ Rsrc buffer_rsrc(const void* base, uint32_t bytes)
{
    const uint64_t a = (uint64_t)(uintptr_t)base;
    Rsrc r;
    r[0] = __builtin_amdgcn_readfirstlane((int32_t)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int32_t)((a >> 32) & 0xFFFFu));
    r[2] = __builtin_amdgcn_readfirstlane((int32_t)bytes);
    r[3] = 0x00020000;  // raw buffer, 32-bit data format
    return r;
}

__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// 64 lanes x 16 (lds_load16) or 4 bytes (lds_load4) from rsrc + voff + soff to
// the 1 KiB (256 bytes) of LDS at byte address lds, lane l's piece at place l.
// Inline assembly, so that the compiler adds no waits of its own before LDS
// reads: whoever reads the data waits on vmcnt and a barrier first, with a
// memory clobber there (none here: LDS reads of other places may pass).
__device__ __forceinline__ void lds_load16(Rsrc rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc),
                 "s"(soff), "s"(lds)
                 : "m0");
}

__device__ __forceinline__ void lds_load4(Rsrc rsrc, uint32_t voff, uint32_t soff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc),
                 "s"(soff), "s"(lds)
                 : "m0");
}

// Waits until at most N of this wave's vector memory operations (loads into
// LDS among them) are unfinished; they finish in order.
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "six bits");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace cmoe
