// lds_load.h -- direct-to-LDS buffer loads for kernels that count their own
// outstanding loads.  Internal to the library.
#pragma once

#include "qmm_internal.h"

namespace qmm {

typedef int ll_i32x4 __attribute__((ext_vector_type(4)));

__device__ inline ll_i32x4 ll_rsrc(const void *base, uint32_t bytes)
{
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return ll_i32x4{(int)(uint32_t)p, (int)((uint32_t)(p >> 32) & 0xFFFFu), (int)bytes, BUFFER_FLAGS};
}

// Written as instructions the compiler does not see, so that it neither moves
// LDS reads across them nor waits for them; lane i of one load writes its SIZE
// bytes at lds + SIZE * i (zeros for an offset out of range).  The consumer
// waits with ll_wait and a barrier.  m0 carries the LDS address; no other code
// of a kernel using these may rely on it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int SIZE>
__device__ inline void ll_load(const ll_i32x4 &rsrc, uint32_t lds, uint32_t voff)
{
    static_assert(SIZE == 4 || SIZE == 16, "dword or dwordx4");
    if constexpr (SIZE == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :: "s"(lds), "v"(voff), "s"(rsrc) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                     :: "s"(lds), "v"(voff), "s"(rsrc) : "memory", "m0");
}
#pragma clang diagnostic pop

// Wait until at most N vector memory operations of this wave are pending.
template <int N>
__device__ inline void ll_wait()
{
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

}  // namespace qmm
