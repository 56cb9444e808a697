// Buffer descriptors and loads from memory straight into LDS, with explicit waits.
#pragma once

#include "common.hpp"

namespace fp8q {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr uint32_t OOB = 0x80000000u;  // an offset past any buffer: loads give zeros, stores are dropped
typedef int i32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4_t make_rsrc4(const void* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)base;  // block-uniform: keep the descriptor in SGPRs
    return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                   __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
                   __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// 16 bytes per lane from a buffer straight into LDS at lds_base + 16*lane (lds_base is
// wave-uniform).  Written as inline assembly so that the compiler does not order every later
// LDS read after it: the waits are explicit (s_waitcnt vmcnt before the step's barrier).
//
// The compiler's hazard pass does not look inside, so each block holds the waits that gfx9 asks for
// and the hardware does not make: one state between the write of M0 and a load to LDS, which takes
// its address from there, and five between a vector instruction that wrote one of the descriptor's or
// the offset's scalar registers (a lane read that fills a descriptor or brings a spilled one back)
// and the load that reads it.  s_mov is one state and s_nop 3 four; the build checks every block.
// Against one state alone: block-scaled 8192 x 14336 x 4096 431 and 423 us, backward of 32 experts of
// 2048 x 7168 807 and 802, others within 1%.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(i32x4_t rsrc, uint32_t voff, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds_base), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
// The same with a wave-uniform offset on top of the lanes'.
__device__ __forceinline__ void dma16_at(i32x4_t rsrc, uint32_t voff, uint32_t soff, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds_base), "v"(voff), "s"(rsrc), "s"(soff)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(i32x4_t rsrc, uint32_t voff, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds_base), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ void wait_vm0() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr_t)p);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                             0x00020000);
}

}  // namespace fp8q
