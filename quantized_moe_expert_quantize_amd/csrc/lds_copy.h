// Copies from global memory into LDS that run beside the kernel's other work, and
// the waits and barriers that go with them.
#pragma once

#include "ftq_internal.h"

namespace ftq {
namespace {

// Asynchronous copies from global memory into LDS, 16 or 4 bytes a lane, to
// consecutive LDS addresses from `lds` (uniform).  Written as asm because the
// compiler, which cannot tell the buffers of successive K blocks apart, would wait
// for a copy in flight before every LDS read; the copies have no result
// registers, and wait_copies() is the only thing that orders them.  The wait states
// that the compiler would put in: one between a write of m0 and the copy, and five
// between a vector instruction's write of a scalar register and a copy that takes
// its address from it.
__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)(const uint8_t*)p;
}
__device__ __forceinline__ void copy16(uint32_t lds, const uint8_t* base, uint32_t off)
{
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void copy16(uint32_t lds, const uint8_t* p)
{
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void copy4(uint32_t lds, const float* p)
{
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void wait_copies() { __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Barrier of the workgroup for LDS alone: global loads stay in flight across it.
__device__ __forceinline__ void block_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// All of the wave's global accesses so far have ended, and the compiler knows it: before a loop that copies, so
// that it puts no wait of its own (which would wait for the copies too) into the loop.
__device__ __forceinline__ void settle() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// At most N of the wave's global accesses are left in flight (they end in their order).
template <int N> __device__ __forceinline__ void wait_copies_but() { __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

}  // namespace
}  // namespace ftq
