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

// A whole warp waits for several phases at once, each lane for its own (none: null): a wait
// costs 150 to 300 cycles even where the phase is long complete, one after the other too many.
__device__ __forceinline__ bool lanes_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* status) {
    if (!__all_sync(0xffffffffu, !bar || mbar_try_wait(bar, parity)) &&
        !__all_sync(0xffffffffu, !bar || wait_or_abort(bar, parity, abort_flag, status)))
        return false;
    __syncwarp();
    return true;
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

// Division by a launch's constant (Granlund and Montgomery, "Division by Invariant Integers using
// Multiplication", 1994; n < 2^31): floor(n / d) = (mulhi(n, m) + n) >> s with
// s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1.  A division proper is a few hundred
// cycles of latency to a lone warp.
struct FastDiv {
    uint32_t d, m, s;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
        while ((uint64_t(1) << s) < d) ++s;
        m = static_cast<uint32_t>((uint64_t(1) << 32) * ((uint64_t(1) << s) - d) / d + 1);
    }
    __host__ __device__ __forceinline__ int div(int n) const {
#ifdef __CUDA_ARCH__
        const uint32_t hi = __umulhi(static_cast<uint32_t>(n), m);
#else
        const uint32_t hi = static_cast<uint32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m) >> 32);
#endif
        return static_cast<int>((hi + static_cast<uint32_t>(n)) >> s);
    }
};

// The work items of a persistent CTA as digits (sequence, tile, part): each step adds the
// grid's digits, with no division.
struct Walk {
    int b, tile, part;
};
struct WalkPlan {
    int batch, tiles, parts;
    Walk step;                                                 // digits of the grid
    __host__ __device__ __forceinline__ Walk at(int item) const {
        const int rest = item / parts;
        return Walk{rest / tiles, rest % tiles, item % parts};
    }
    __device__ __forceinline__ bool in(const Walk& w) const { return w.b < batch; }
    __device__ __forceinline__ void next(Walk& w) const {
        w.part += step.part;
        w.tile += step.tile;
        w.b += step.b;
        if (w.part >= parts) { w.part -= parts; ++w.tile; }
        if (w.tile >= tiles) { w.tile -= tiles; ++w.b; }
    }
};

}  // namespace hs2
