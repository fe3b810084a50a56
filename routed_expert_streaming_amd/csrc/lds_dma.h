// Direct global -> LDS loads, the waits and the barrier that go with a ring of them, and
// what the matrix kernels share beside them.
#pragma once
#include "common.h"

typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ uint32_t lds_addr(const void *lds) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_u8 *)lds);
}
// Direct global->LDS load: lane l's 16 bytes from base + off land at LDS byte lds +
// 16*l (lds uniform; base uniform, in SGPRs; off this lane's 32-bit byte offset).
// Written as inline asm because the compiler, seeing these loads, would make every
// later LDS read wait for all of them (it cannot tell a ring's stages apart);
// completion is tracked with explicit vmcnt waits instead (a wave's loads complete
// in order).  The memory clobber keeps the compiler's own loads in program order
// around it, which the wait counts rely on.
// The s_nop gives the 5 wait states a vector memory instruction needs after a
// VALU instruction wrote an SGPR it reads (and the one after an M0 write): the
// compiler inserts these for its own instructions but cannot see into inline
// asm, and under register pressure it restores a spilled base half with
// v_readlane right before the load -- without the wait the load can use the
// stale half and go to a wrong address.
__device__ __forceinline__ void dma16(const void *base, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}

// Waits until at most N of the wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup barrier without a memory fence (a fence would wait for every load
// in flight); this wave's LDS accesses are done when it arrives.
__device__ __forceinline__ void ring_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int N>
struct IntC {
    static constexpr int value = N;
};

// f(IntC<B>{}), f(IntC<B + 1>{}), ..., f(IntC<E - 1>{})
template <int B, int E, class F>
__device__ __forceinline__ void static_for(F &&f) {
    if constexpr (B < E) {
        f(IntC<B>{});
        static_for<B + 1, E>(f);
    }
}

// Two floats -> bf16 pair, rounded to nearest even, lo in bits 0-15 (one instruction).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(
        uint32_t, __builtin_convertvector((float __attribute__((ext_vector_type(2)))){lo, hi}, moe_bf16x2));
}
