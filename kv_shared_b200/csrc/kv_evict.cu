// kv_evict.cu -- eviction from a cache by accumulated attention weight.
//
// Of a sequence's n rows the first `sinks`, the latest `window` and the `budget` largest
// totals between them survive, in order.  Two launches:
//
//   select  The totals' bit patterns, made to order like the values, are counted by their upper
//           11 bits, and the digit in which the budget runs out follows; the middle 11 and the
//           lower 10 bits are found the same way among the rows that share the bits so far.
//           With the exact threshold pattern T and how many equal to it are still wanted (the
//           lowest rows), a last pass writes the survivors' rows in order.  No atomic decides a
//           position, so equal calls give equal bits.  A sequence is one CTA's, a cluster's
//           (counts added through distributed shared memory) or, where clusters leave SMs idle,
//           that of a team of SMs / batch CTAs that meet in grid-wide barriers (a cooperative
//           launch; their counts meet in the sequence's rows of k_out, which the move then
//           overwrites).  The patterns stay in shared memory; slices too long for it (many
//           sequences, each over 40960 rows a CTA) are read again, and only the rows that share
//           the first digit are listed.
//   move    one warp per few rows copies K, V, scales and totals to their new places, and one thread
//           per sequence writes the new length: every CTA of the selection has read the old one by
//           then, so that lengths may be cut in place.
//
// The move is bound by HBM (twice the surviving rows' bytes; the kernel alone: 525,000 e4m3 rows 50 us,
// 32 x 4228 bf16 rows 24.6 us), the selection by its barriers (5 to 9 us for one CTA, 22 us for 1M rows or
// 32 x 64K).  Times below are of whole calls replayed from a graph on the same inputs; among other
// calls, on changing inputs, 1M e4m3 rows halved take 77.4 us and 32 x 64K bf16 rows 51.7.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace hs2 {
namespace {

constexpr int ST = 1024;                         // threads of a select CTA
constexpr int SW = ST / 32;
constexpr int BINS = 2048;
constexpr int COPIES = 4;                        // of the first round's counts (warps share them in turn)
// rows per sequence up to which one CTA selects (1 x 4000: 11.6 us against a cluster's 17.0;
// 4 x 16384: 17.9 against 18.2, 1 x 20000: 18.8 against 17.2)
constexpr int64_t kOneRows = 16384;
constexpr int kMaxCluster = 16;                  // more than 8 is an opt-in
constexpr int LIST = 12288;                      // rows of a CTA's slice in the threshold's digit
constexpr int LD = 16;                           // totals in flight per lane
constexpr int kSelectSmem = (COPIES * BINS + BINS) * 4 + LIST * 8;

// Bits that order like the values: -0 as 0, a NaN below everything.
__device__ __forceinline__ uint32_t order_bits(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);                // -0 + 0 = 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A lane's LD totals 32 apart from position i on (0 from `end` on).
__device__ __forceinline__ void load_part(const float* acc, int i, int end, float (&x)[LD]) {
#pragma unroll
    for (int j = 0; j < LD; ++j) x[j] = i + 32 * j < end ? __ldg(acc + i + 32 * j) : 0.f;
}

// Sum over the threads before this one; *total: over all (ST threads; scratch [SW + 1]).
__device__ __forceinline__ int block_scan(int v, int* scratch, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                                            // scratch is free
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = scratch[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        scratch[lane] = w;
    }
    __syncthreads();
    *total = scratch[SW - 1];
    return x - v + (warp ? scratch[warp - 1] : 0);
}

__global__ void __launch_bounds__(ST) evict_select_kernel(EvictArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = static_cast<int>(cluster.num_blocks()), cr = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / cs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    extern __shared__ int dyn[];
    int* hist = dyn;                                            // [COPIES][BINS]
    int* sums = hist + COPIES * BINS;                           // [BINS] over the cluster
    uint2* list = reinterpret_cast<uint2*>(sums + BINS);        // [LIST] (pattern, row of the slice)
    __shared__ int scratch[SW + 1];
    __shared__ int digit, rest, listed, count2[2];
    __shared__ int before2[2];
    __shared__ int warp_gt[SW], warp_eq[SW];

    const int64_t keep = static_cast<int64_t>(a.sinks) + a.window + a.budget;
    int64_t n64 = a.len[b];
    n64 = n64 < 0 ? 0 : (n64 > a.cap ? a.cap : n64);
    const int n = static_cast<int>(n64);
    const int kept = n < keep ? n : static_cast<int>(keep);
    int32_t* idx = a.idx + b * keep;
    for (int64_t i = kept + cr * ST + tid; i < keep; i += cs * ST) idx[i] = -1;
    if (n <= keep) {                                            // the whole cluster takes this branch
        for (int i = cr * ST + tid; i < n; i += cs * ST) idx[i] = i;
        return;
    }
    const int first = a.sinks, m = n - a.window - a.sinks;      // candidates first .. first + m - 1, m > budget
    for (int i = cr * ST + tid; i < a.sinks; i += cs * ST) idx[i] = i;
    for (int i = cr * ST + tid; i < a.window; i += cs * ST) idx[a.sinks + a.budget + i] = n - a.window + i;
    if (a.budget == 0) return;

    // this CTA's slice of the candidates, and each warp's part of it
    const int per = (m + cs - 1) / cs;
    const int lo = min(m, cr * per), hi = min(m, lo + per);
    const int seg = ((hi - lo + SW - 1) / SW + 31) & ~31;       // whole warps wide
    const int s0 = min(hi, lo + warp * seg), s1 = min(hi, s0 + seg);
    const float* acc = a.acc + b * a.cap + first;

    uint32_t prefix = 0;                                        // bits of T found so far
    int want = a.budget;                                        // still wanted among those that share them
    int gt = 0;                                                 // of this lane, above the first digit
    bool use_list = true;
    if (tid < SW) warp_gt[tid] = warp_eq[tid] = 0;
    if (tid == 0) listed = 0;
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
        const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0);
        const uint32_t mask = round == 2 ? 1023u : 2047u;
        const uint32_t above = round == 0 ? 0u : (round == 1 ? 0xffe00000u : 0xfffffc00u);
        const int copies = round == 0 ? COPIES : 1;
        for (int i = tid; i < copies * BINS; i += ST) hist[i] = 0;
        __syncthreads();
        if (round == 0) {
            int* mine = hist + (warp % COPIES) * BINS;
            for (int i0 = s0; i0 < s1; i0 += 32 * LD) {
                float x[LD];
                load_part(acc, i0 + lane, s1, x);
#pragma unroll
                for (int j = 0; j < LD; ++j)
                    if (i0 + 32 * j + lane < s1) atomicAdd(&mine[order_bits(x[j]) >> 21], 1);
            }
            __syncthreads();
            for (int i = tid; i < BINS; i += ST) {
                int c = hist[i];
#pragma unroll
                for (int k = 1; k < COPIES; ++k) c += hist[k * BINS + i];
                hist[i] = c;
            }
        } else if (round == 1) {
            // above the digit: counted; in it: listed, and counted by the next digit
            for (int i0 = s0; i0 < s1; i0 += 32 * LD) {
                float x[LD];
                load_part(acc, i0 + lane, s1, x);
#pragma unroll
                for (int j = 0; j < LD; ++j) {
                    const int i = i0 + 32 * j + lane;
                    const uint32_t u = order_bits(x[j]);
                    const bool in = i < s1, tie = in && (u & above) == prefix;
                    gt += in && (u & above) > prefix;
                    if (tie) atomicAdd(&hist[(u >> shift) & mask], 1);
                    const uint32_t mt = __ballot_sync(0xffffffffu, tie);
                    if (mt) {
                        int at = 0;
                        if (lane == 0) at = atomicAdd(&listed, __popc(mt));
                        at = __shfl_sync(0xffffffffu, at, 0) + __popc(mt & ((1u << lane) - 1u));
                        if (tie && at < LIST) list[at] = make_uint2(u, static_cast<uint32_t>(i - lo));
                    }
                }
            }
            __syncthreads();
            use_list = listed <= LIST;                          // the same in every thread of the CTA
        } else if (use_list) {
            for (int i = tid; i < listed; i += ST) {
                const uint32_t u = list[i].x;
                if ((u & above) == prefix) atomicAdd(&hist[u & mask], 1);
            }
        } else {
            for (int i0 = s0; i0 < s1; i0 += 32 * LD) {
                float x[LD];
                load_part(acc, i0 + lane, s1, x);
#pragma unroll
                for (int j = 0; j < LD; ++j) {
                    const uint32_t u = order_bits(x[j]);
                    if (i0 + 32 * j + lane < s1 && (u & above) == prefix) atomicAdd(&hist[u & mask], 1);
                }
            }
        }
        cluster.sync();
        // every CTA adds up its share of the bins over the cluster and hands the sums to all
        const int share = BINS / cs;
        for (int i = tid; i < share; i += ST) {
            const int bin = cr * share + i;
            int s = 0;
            for (int r = 0; r < cs; ++r) s += cluster.map_shared_rank(hist, r)[bin];
            for (int r = 0; r < cs; ++r) cluster.map_shared_rank(sums, r)[bin] = s;
        }
        cluster.sync();
        // the digit in which the budget runs out, from the highest down: thread t has the bins
        // 2047 - 2t and 2046 - 2t
        const int c0 = sums[BINS - 1 - 2 * tid], c1 = sums[BINS - 2 - 2 * tid];
        int total;
        const int over = block_scan(c0 + c1, scratch, &total);
        if (over < want && over + c0 >= want) { digit = BINS - 1 - 2 * tid; rest = want - over; }
        else if (over + c0 < want && over + c0 + c1 >= want) { digit = BINS - 2 - 2 * tid; rest = want - over - c0; }
        __syncthreads();
        prefix |= static_cast<uint32_t>(digit) << shift;
        want = rest;
        __syncthreads();
    }
    // T = prefix; of the rows equal to it the first `want` are kept.  Per warp: rows above T and
    // equal to it.
    int eq = 0;
    if (use_list) {
        for (int i = tid; i < listed; i += ST) {
            const uint2 e = list[i];
            if (e.x > prefix) atomicAdd(&warp_gt[e.y / seg], 1);
            else if (e.x == prefix) atomicAdd(&warp_eq[e.y / seg], 1);
        }
    } else {
        gt = 0;
        for (int i0 = s0; i0 < s1; i0 += 32 * LD) {
            float x[LD];
            load_part(acc, i0 + lane, s1, x);
#pragma unroll
            for (int j = 0; j < LD; ++j) {
                const bool in = i0 + 32 * j + lane < s1;
                const uint32_t u = order_bits(x[j]);
                gt += in && u > prefix;
                eq += in && u == prefix;
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        gt += __shfl_xor_sync(0xffffffffu, gt, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    __syncthreads();
    gt += warp_gt[warp];
    eq += warp_eq[warp];
    int gt_all, eq_all;
    int gt_at = block_scan(lane == 0 ? gt : 0, scratch, &gt_all);
    int eq_at = block_scan(lane == 0 ? eq : 0, scratch, &eq_all);
    if (tid == 0) { count2[0] = gt_all; count2[1] = eq_all; }
    cluster.sync();
    if (tid < 2) {
        int s = 0;
        for (int r = 0; r < cr; ++r) s += cluster.map_shared_rank(count2, r)[tid];
        before2[tid] = s;
    }
    cluster.sync();                                             // also: no CTA leaves while it is read
    gt_at = __shfl_sync(0xffffffffu, gt_at, 0) + before2[0];
    eq_at = __shfl_sync(0xffffffffu, eq_at, 0) + before2[1];
    const uint32_t lt = (1u << lane) - 1u;
    for (int i0 = s0; i0 < s1; i0 += 32 * LD) {
        float x[LD];
        load_part(acc, i0 + lane, s1, x);
#pragma unroll
        for (int j = 0; j < LD; ++j) {
            const int i = i0 + 32 * j + lane;
            const uint32_t u = order_bits(x[j]);
            const uint32_t mg = __ballot_sync(0xffffffffu, i < s1 && u > prefix);
            const uint32_t me = __ballot_sync(0xffffffffu, i < s1 && u == prefix);
            const int g = gt_at + __popc(mg & lt), e = eq_at + __popc(me & lt);
            if (((mg >> lane) & 1u) || (((me >> lane) & 1u) && e < want)) idx[first + g + min(e, want)] = first + i;
            gt_at += __popc(mg);
            eq_at += __popc(me);
        }
    }
}

// The same with the slices' patterns in shared memory, by `team` CTAs per sequence: one (ONE), a
// cluster, or any number that meets in grid-wide barriers (GRID).
constexpr int kKeys = 40960;                     // rows of a CTA's slice, at most
constexpr int team_smem(int64_t slice) { return static_cast<int>((COPIES * BINS + BINS + slice) * 4); }
constexpr int kTeamSmem = team_smem(kKeys);
constexpr int kScratchInts = 3 * BINS;           // GRID: counts of the three rounds; then two per CTA
enum { ONE = 0, CLUSTER = 1, GRID = 2 };

template <int MODE>
__global__ void __launch_bounds__(ST) evict_team_kernel(EvictArgs a, int team, int row_bytes) {
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.x / team, tr = blockIdx.x - b * team;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    extern __shared__ int dyn[];
    int* hist = dyn;                                            // [COPIES][BINS]
    int* sums = hist + COPIES * BINS;                           // [BINS] over the team
    uint32_t* keys = reinterpret_cast<uint32_t*>(sums + BINS);  // [slice]
    __shared__ int scratch[SW + 1];
    __shared__ int digit, rest, count2[2], before2[2];

    const int64_t keep = static_cast<int64_t>(a.sinks) + a.window + a.budget;
    int64_t n64 = a.len[b];
    n64 = n64 < 0 ? 0 : (n64 > a.cap ? a.cap : n64);
    const int n = static_cast<int>(n64);
    const int kept = n < keep ? n : static_cast<int>(keep);
    int32_t* idx = a.idx + b * keep;
    const bool cut = n > keep && a.budget > 0;                  // the same in the whole team
    const int first = a.sinks, m = cut ? n - a.window - a.sinks : 0;
    const int per = (m + team - 1) / team;
    const int lo = min(m, tr * per), mine = min(m, lo + per) - lo;
    const float* acc = a.acc + b * a.cap + first + lo;
    // GRID: the sequence's rows of k_out, only where rows are cut, hence all of them written later
    int* counts = reinterpret_cast<int*>(static_cast<uint8_t*>(a.k_out) + static_cast<int64_t>(b) * a.out_cap * row_bytes);
    for (int i = tid; i < COPIES * BINS; i += ST) hist[i] = 0;
    if (MODE == GRID && cut)
        for (int i = tr * ST + tid; i < kScratchInts; i += team * ST) counts[i] = 0;
    __syncthreads();
    int* copy = hist + (warp % COPIES) * BINS;
    for (int i0 = 0; i0 < mine; i0 += ST * 8) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = i0 + j * ST + tid < mine ? __ldg(acc + i0 + j * ST + tid) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + j * ST + tid < mine) {
                const uint32_t u = order_bits(x[j]);
                keys[i0 + j * ST + tid] = u;
                atomicAdd(&copy[u >> 21], 1);
            }
    }
    // what does not depend on the totals
    for (int64_t i = kept + tr * ST + tid; i < keep; i += team * ST) idx[i] = -1;
    if (n <= keep) {
        for (int i = tr * ST + tid; i < n; i += team * ST) idx[i] = i;
    } else {
        for (int i = tr * ST + tid; i < a.sinks; i += team * ST) idx[i] = i;
        for (int i = tr * ST + tid; i < a.window; i += team * ST) idx[a.sinks + a.budget + i] = n - a.window + i;
    }
    if (MODE != GRID && !cut) return;                           // the whole team
    __syncthreads();
    if (MODE == GRID) cg::this_grid().sync();                   // the counts are zero
    uint32_t prefix = 0;                                        // bits of T found so far
    int want = a.budget;                                        // still wanted among those that share them
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
        const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0);
        const uint32_t mask = round == 2 ? 1023u : 2047u;
        const uint32_t above = round == 0 ? 0u : (round == 1 ? 0xffe00000u : 0xfffffc00u);
        if (round > 0) {
            for (int i = tid; i < BINS; i += ST) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < mine; i += ST) {
                const uint32_t u = keys[i];
                if ((u & above) == prefix) atomicAdd(&hist[(u >> shift) & mask], 1);
            }
            __syncthreads();
        }
        for (int i = tid; i < BINS; i += ST) {
            int c = hist[i];
            if (round == 0)
#pragma unroll
                for (int k = 1; k < COPIES; ++k) c += hist[k * BINS + i];
            if (MODE == ONE) sums[i] = c;
            else if (MODE == CLUSTER) hist[i] = c;
            else if (cut && c) atomicAdd(&counts[round * BINS + i], c);
        }
        if (MODE == ONE) {
            __syncthreads();
        } else if (MODE == CLUSTER) {
            cluster.sync();
            // every CTA adds up its share of the bins over the cluster and hands the sums to all
            const int share = BINS / team;
            for (int i = tid; i < share; i += ST) {
                const int bin = tr * share + i;
                int c = 0;
                for (int r = 0; r < team; ++r) c += cluster.map_shared_rank(hist, r)[bin];
                for (int r = 0; r < team; ++r) cluster.map_shared_rank(sums, r)[bin] = c;
            }
            cluster.sync();
        } else {
            cg::this_grid().sync();
        }
        if (cut) {
            // the digit in which the budget runs out, from the highest down: thread t has the bins
            // 2047 - 2t and 2046 - 2t
            const int at = BINS / 2 - 1 - tid;
            const int2 c = MODE == GRID ? __ldcg(reinterpret_cast<const int2*>(counts + round * BINS) + at)
                                        : reinterpret_cast<const int2*>(sums)[at];
            int total;
            const int over = block_scan(c.x + c.y, scratch, &total);
            if (over < want && over + c.y >= want) { digit = BINS - 1 - 2 * tid; rest = want - over; }
            else if (over + c.y < want && over + c.y + c.x >= want) { digit = BINS - 2 - 2 * tid; rest = want - over - c.y; }
            __syncthreads();
            prefix |= static_cast<uint32_t>(digit) << shift;
            want = rest;
            __syncthreads();
        }
    }
    // rows above T = prefix and equal to it (the first `want` of which are kept): of this warp's
    // part of the slice, of the CTA, of the CTAs before
    const int seg = ((mine + SW - 1) / SW + 31) & ~31;          // whole warps wide
    const int s0 = min(mine, warp * seg), s1 = min(mine, s0 + seg);
    int gt = 0, eq = 0;
    for (int i = s0 + lane; i < s1; i += 32) {
        const uint32_t u = keys[i];
        gt += u > prefix;
        eq += u == prefix;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        gt += __shfl_xor_sync(0xffffffffu, gt, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    int gt_all, eq_all;
    int gt_at = block_scan(lane == 0 ? gt : 0, scratch, &gt_all);
    int eq_at = block_scan(lane == 0 ? eq : 0, scratch, &eq_all);
    gt_at = __shfl_sync(0xffffffffu, gt_at, 0);
    eq_at = __shfl_sync(0xffffffffu, eq_at, 0);
    if (MODE != ONE) {
        int* team2 = counts + kScratchInts;                     // GRID: [team][2]
        if (cut && tid == 0) {
            if (MODE == GRID) { team2[2 * tr] = gt_all; team2[2 * tr + 1] = eq_all; }
            else { count2[0] = gt_all; count2[1] = eq_all; }
        }
        if (MODE == GRID) cg::this_grid().sync();
        else cluster.sync();
        if (!cut) return;
        if (warp < 2) {
            int c = 0;
            for (int r = lane; r < tr; r += 32)
                c += MODE == GRID ? __ldcg(team2 + 2 * r + warp) : cluster.map_shared_rank(count2, r)[warp];
#pragma unroll
            for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            if (lane == 0) before2[warp] = c;
        }
        if (MODE == CLUSTER) cluster.sync();                    // also: no CTA leaves while it is read
        else __syncthreads();
        gt_at += before2[0];
        eq_at += before2[1];
    }
    const uint32_t lt = (1u << lane) - 1u;
    for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t u = i < s1 ? keys[i] : 0u;
        const uint32_t mg = __ballot_sync(0xffffffffu, i < s1 && u > prefix);
        const uint32_t me = __ballot_sync(0xffffffffu, i < s1 && u == prefix);
        const int g = gt_at + __popc(mg & lt), e = eq_at + __popc(me & lt);
        if (((mg >> lane) & 1u) || (((me >> lane) & 1u) && e < want)) idx[first + g + min(e, want)] = first + lo + i;
        gt_at += __popc(mg);
        eq_at += __popc(me);
    }
}

// Rows to their new places.  ROW: bytes of a K (V) row; 16 bytes per lane, 512 / ROW rows of K
// and V each per step of a warp, UN steps in flight.
template <int ROW>
__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a, int64_t keep, int blocks) {
    constexpr int LPR = ROW / 16;                               // lanes per row
    constexpr int RPS = LPR > 32 ? 0 : 32 / LPR;                // rows per step
    constexpr int UN = 4;
    static_assert(RPS >= 1, "a row spans at most a warp");
    const int b = blockIdx.x / blocks;
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x - b * blocks) * 8 + (threadIdx.x >> 5);
    const int64_t r0 = w * RPS * UN;
    if (w == 0 && lane == 0) {
        const int64_t n = min(max(static_cast<int64_t>(a.len[b]), int64_t(0)), a.cap);
        a.new_len[b] = static_cast<int32_t>(min(n, keep));
    }
    const int32_t* idx = a.idx + b * keep;
    const uint4* k = static_cast<const uint4*>(a.k) + b * a.cap * LPR;
    const uint4* v = static_cast<const uint4*>(a.v) + b * a.cap * LPR;
    uint4* ko = static_cast<uint4*>(a.k_out) + b * a.out_cap * LPR;
    uint4* vo = static_cast<uint4*>(a.v_out) + b * a.out_cap * LPR;
    const int c = lane % LPR;
    int src[UN];
    uint4 kx[UN], vx[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        const int64_t r = r0 + u * RPS + lane / LPR;
        src[u] = r < keep ? __ldg(idx + r) : -1;
    }
#pragma unroll
    for (int u = 0; u < UN; ++u)
        if (src[u] >= 0) {
            kx[u] = __ldg(k + static_cast<int64_t>(src[u]) * LPR + c);
            vx[u] = __ldg(v + static_cast<int64_t>(src[u]) * LPR + c);
        }
#pragma unroll
    for (int u = 0; u < UN; ++u)
        if (src[u] >= 0) {
            const int64_t r = r0 + u * RPS + lane / LPR;
            ko[r * LPR + c] = kx[u];
            vo[r * LPR + c] = vx[u];
            if (c == 0) {
                const int64_t s = b * a.cap + src[u], d = b * a.out_cap + r;
                if (a.acc_out) a.acc_out[d] = __ldg(a.acc + s);
                if (a.kv_dtype == HS2_E4M3) {
                    a.k_scale_out[d] = __ldg(a.k_scale + s);
                    a.v_scale_out[d] = __ldg(a.v_scale + s);
                }
            }
        }
}

template <int ROW>
void move(const EvictArgs& a, int64_t keep, cudaStream_t st) {
    constexpr int rows = 8 * 4 * (32 / (ROW / 16));             // per CTA
    const int blocks = static_cast<int>((keep + rows - 1) / rows);
    evict_move_kernel<ROW><<<static_cast<unsigned>(blocks) * a.batch, 256, 0, st>>>(a, keep, blocks);
}

// CTAs per sequence of a cluster: as many as keep the batch on the SMs at once, up to the
// largest cluster, and no more than leaves each a few thousand rows.
int cluster_size(const EvictArgs& a) {
    int cs = 1;
    while (cs < kMaxCluster && 2 * cs * a.batch <= num_sms() && a.cap > static_cast<int64_t>(cs) * 4096) cs *= 2;
    return cs;
}

// `most`: the largest smem that any call gives the kernel.  The limit belongs to the function in the
// whole process, so every call sets the same one (a call's own size, set by another thread between this
// thread's set and its launch, made the launch fail).
template <typename Kernel, typename... Args>
cudaError_t launch_select(Kernel kernel, int grid, int smem, int most, cudaLaunchAttribute at, cudaStream_t st, Args... args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(ST);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t select(const EvictArgs& a, int64_t keep, int row, cudaStream_t st) {
    cudaLaunchAttribute cluster{}, coop{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    coop.id = cudaLaunchAttributeCooperative;
    coop.val.cooperative = 1;
    if (a.cap <= kOneRows) {
        cluster.val.clusterDim.x = 1;
        return launch_select(evict_team_kernel<ONE>, a.batch, team_smem(a.cap), kTeamSmem, cluster, st, a, 1, row);
    }
    // Teams of all SMs where a cluster's slices are long and SMs idle, or where large clusters do
    // not all fit at once (a GPC takes one or two of 8), unless k_out has no room for their counts.
    // Measured, the whole call, teams against clusters: 1 x 1M e4m3 rows 74 us against 108, 2 x 256K
    // bf16 43.5 against 45.4, 8 x 128K 47 against 60, 16 x 32K 44 against 52; the other way
    // 1 x 64K 21.7 against 19.6, 4 x 64K 23.2 against 21.5, 32 x 32K 26.6 against 21.9.
    const int team = num_sms() / a.batch, cs = cluster_size(a);
    const int64_t slice = team > 0 ? (a.cap + team - 1) / team : a.cap;
    const bool idle = team >= 2 * cs && a.cap > static_cast<int64_t>(cs) * 8192, crowd = cs >= 8 && a.batch * cs > 64;
    if (team > 1 && slice <= kKeys && (idle || crowd) &&
        keep * row >= 4 * (kScratchInts + 2 * static_cast<int64_t>(team)))
        return launch_select(evict_team_kernel<GRID>, a.batch * team, team_smem(slice), kTeamSmem, coop, st, a, team, row);
    cluster.val.clusterDim.x = cs;
    const int64_t part = (a.cap + cs - 1) / cs;
    if (part <= kKeys)
        return launch_select(evict_team_kernel<CLUSTER>, a.batch * cs, team_smem(part), kTeamSmem, cluster, st, a, cs, row);
    return launch_select(evict_select_kernel, a.batch * cs, kSelectSmem, kSelectSmem, cluster, st, a);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
    const int64_t keep = static_cast<int64_t>(a.sinks) + a.window + a.budget;
    const int row = a.head_dim * (a.kv_dtype == HS2_F32 ? 4 : (a.kv_dtype == HS2_BF16 ? 2 : 1));
    const cudaError_t e = select(a, keep, row, st);
    if (e != cudaSuccess) return e;
    if (row == 64) move<64>(a, keep, st);
    else if (row == 128) move<128>(a, keep, st);
    else if (row == 256) move<256>(a, keep, st);
    else move<512>(a, keep, st);
    return cudaGetLastError();
}

}  // namespace hs2
