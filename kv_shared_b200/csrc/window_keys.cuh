// window_keys.cuh -- which cache rows a tile of consecutive query rows attends to under a
// sliding window with sinks, shared by the window-attention kernels.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace hs2 {

// Rows of sequence b in use, and the position of its first row, moved (and reported) so
// that every position lies in [0, max_ctx).
__device__ __forceinline__ int live_rows(const int32_t* n_rows, int b, int n_q) {
    return n_rows ? min(max(n_rows[b], 0), n_q) : n_q;
}
__device__ __forceinline__ int checked_base(const int32_t* q_pos0, int b, int live, int64_t max_ctx, uint32_t* status) {
    const int p0 = q_pos0[b];
    const int64_t top = max_ctx - live;          // >= 0: live <= n_q <= max_ctx
    if (p0 < 0 || p0 > top) {
        set_status(status, HS2_ERR_INDEX);
        return p0 < 0 ? 0 : static_cast<int>(top);
    }
    return p0;
}

// The union of the rows that positions p_lo .. p_hi attend to, as one list: the sinks that
// lie before the window's range, padded to a multiple of kSinkPad, then the rows lo .. p_hi.
struct KeyList {
    int lo, s_eff, s_pad, total;
    __device__ __forceinline__ KeyList(int p_lo, int p_hi, int window, int sinks) {
        lo = max(0, p_lo - window + 1);
        s_eff = 0;
        if (lo > 0) {
            if (sinks >= lo) lo = 0;
            else s_eff = sinks;
        }
        s_pad = (s_eff + kSinkPad - 1) / kSinkPad * kSinkPad;
        total = s_pad + (p_hi - lo + 1);
    }
    // cache row of list entry u, -1 for padding and entries past the end
    __device__ __forceinline__ int row(int u) const {
        if (u < s_pad) return u < s_eff ? u : -1;
        return u < total ? lo + (u - s_pad) : -1;
    }
};

__device__ __forceinline__ bool window_sees(int key, int p, int window, int sinks) {
    return key >= 0 && key <= p && (key > p - window || key < sinks);
}

}  // namespace hs2
