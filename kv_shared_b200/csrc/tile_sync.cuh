// tile_sync.cuh -- waits and warp helpers of the warp-specialised tcgen05 kernels around the
// block (window_tile.cu, accum_tile.cu).
#pragma once

#include "common.cuh"

namespace hs2 {

// Bounded wait (kWaitNs in all); false, the status word and the CTA's abort flag set, if the
// phase does not complete in time, and false at once where another role has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
    if (*abort_flag) return false;
    if (!mbar_wait(bar, parity, status)) { *abort_flag = 1; return false; }
    return true;
}
// The same for a whole warp; in the common case, without a look at the flag or the clock.
// (try_wait's own short suspensions measured best: polled with test_wait or suspended for
// 20 us at a time the kernels were 4 to 17% slower.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, status));
}

// One lane of a converged warp, the same every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// The warp's common value in a uniform register (a reduction leaves it there).
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// The lowest n bits.
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

}  // namespace hs2
