// tcgen05_epilogue.cuh -- what the epilogues of the 8-bit and adapter products
// need beside tcgen05.cuh: narrow TMEM loads, and waits of warps in turns.
#pragma once
#include "tcgen05.cuh"

namespace qlora {
namespace tc {

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

// One turn of THREADS threads that meet at a named barrier and then wait for
// `bar`.  A warp whose wait has given up (ok false) goes on meeting the others
// turn after turn without waiting again: they may not have given up, and a
// barrier that a warp has left never fills.
template <int BARRIER, int THREADS>
__device__ __forceinline__ bool mbar_wait_turn(bool ok, uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    asm volatile("bar.sync %0, %1;\n" ::"n"(BARRIER), "n"(THREADS) : "memory");
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort_flag));
    if (!ok) *abort_flag = 1;
    return ok;
}

}  // namespace tc
}  // namespace qlora
