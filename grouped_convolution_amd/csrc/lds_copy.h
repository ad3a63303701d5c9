// lds_copy.h -- copies from global memory straight to LDS, and the wait for them,
// for kernels that keep a ring of stages under way.
#pragma once

#include "seq_util.h"

namespace gconv {

typedef __attribute__((address_space(3))) char lds_char;

// 64 lanes' 16 bytes from global memory straight to 1024 bytes of LDS. In
// assembly, as it writes no register: the compiler would otherwise wait for
// every such load before any read of LDS, where the stages below wait once. M0
// is said to be written, and no one needs it kept, which is what the compiler
// warns of.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_lds(u4 rsrc, uint32_t lds, uint32_t off)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(off), "s"(rsrc) : "memory", "m0");
}
#pragma clang diagnostic pop

// Waits until at most N of this wave's loads are still under way.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

__device__ __forceinline__ u4 resource(const void* p, uint32_t bytes)
{
    const uint64_t v = (uint64_t)p;
    return u4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v), (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)),
              (uint32_t)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
}

}  // namespace gconv
