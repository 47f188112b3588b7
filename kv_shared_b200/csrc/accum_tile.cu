// accum_tile.cu -- accumulated attention weight of the cached keys on tcgen05, for bf16 and
// e4m3 caches.
//
//   acc_out[j] = decay acc_in[j] + sum over rows r and heads h of
//                exp(scale q_rh . k_j - lse_rh)            [j <= p_r]
//
// The log-sum-exp is known, so there is nothing to carry from key to key: S = K Q^T with the
// keys in the MMA's M dimension puts a key's logits into one tensor-memory lane, and its total
// is a sum inside a thread.  A CTA holds a block of keys in shared memory and streams the
// (row, head) pairs past it, so each key is read from HBM once and each Q tile from L2 once
// per block.  Long calls are bound by the exponential unit (one exponential per key and pair,
// 8 cycles a warp; an eighth of them moves to the FMA pipe), calls of a few pairs by the read of K.
//
// Two shapes of a work item (sequence, key block, part of the pairs):
//   wide   2 x 128 keys, pairs in tiles of 128; two teams of warps take the tiles in turn, so
//          that one's handovers fall into the other's exponentials (with both on the same
//          tile, 64 columns a thread, everything waited at once: 3300 cycles a tile)
//   narrow 4 x 128 keys, all pairs in one tile of at most 64 columns (single tokens): a thread
//          per key, so that no thread idles and an item is worth its handovers
// S is double-buffered (2 x 256 columns of tensor memory): the MMAs of the next tile run
// while the exponentials of this one are formed.
//
// e4m3 caches: the codes are the MMA's operand as they lie in the cache.  Q goes in as a sum of
// two e4m3 numbers, found once per call: q 2^e = hi + lo with the row's largest magnitude in
// [128, 256).  bf16 has 8 significant bits and e4m3 4, so hi takes the upper and lo the lower
// ones exactly, down to elements 2^-9 of the row's largest; smaller ones are rounded to 2^-17
// of it at worst.
//
// Measured, replayed from a graph on the same inputs: 32 rows of 16 heads over 4 x 131072 bf16
// keys 92 us (750 TFLOP/s; exponentials and their arithmetic alone would take 50), one row over
// 8 x 100001 e4m3 keys 25.5 us (4.3 TB/s).  As calls among others on changing inputs: 104.6 and 28.5.
//
// Roles (640 threads): warps 0-15 exponentials, 16 the TMA loads, 17 the pairs' lse (and
// scales), 18 and 19 the MMAs of the even and the odd 128 keys.  Every wait is bounded; a
// wait that gives up flags the status word and makes all roles leave their loops.
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "tile_sync.cuh"
#include "window_keys.cuh"

namespace hs2 {
namespace {

constexpr int NT = 640;
constexpr int NEXP = 16;                        // exponential warps
constexpr int MK = 128;                         // keys per MMA
constexpr int NL = 4;                           // tiles whose lse are held
constexpr int kNarrow = 64;                     // most pairs of the narrow shape
// Of 8 groups of 4 columns: which take the FMA pipe.  Two of them need more instructions than the
// exponential unit saves: 32 rows of 16 heads over 4 x 131072 keys, bf16 and e4m3, 104 and 116 us a call,
// one 102 and 113.
constexpr uint32_t kPolyGroups = 0x01;
constexpr int kSmem = 232448;
constexpr int kBars = 16 + 16 + 4 + 4 + 8 + 8 + NL + NL + 8;
constexpr int OFF_XCH = 1024, OFF_NL = OFF_XCH + 4 * 2 * MK * 4, OFF_TILES = OFF_NL + NL * 2 * MK * 4;
static_assert(kBars * 8 + 8 <= OFF_XCH && OFF_TILES % 1024 == 0, "control block");

struct TileArgs {
    AccumArgs a;
    WalkPlan walk;                              // (sequence, key block, part of the pairs)
    bool narrow;
    int n_cols;                                 // pairs per Q tile (a multiple of 16)
    int k_stages, q_slots, q_bytes;
    const float* q_scale;                       // e4m3: 2^-e of each pair
};

template <int D, bool KV8>
struct Shape {
    static constexpr int ROW = KV8 ? D : 2 * D;                // bytes of a K row
    static constexpr int KBOX = ROW < 128 ? ROW : 128;         // bytes of a swizzled box's row
    static constexpr int KBOXES = ROW / KBOX;
    static constexpr int KTILE = MK * ROW;
    // Q rows: bf16 in 64-column boxes; e4m3 hi then lo, a box each
    static constexpr int QBOXES = KV8 ? 2 : D / 64;
    static constexpr int QROW = 2 * D;
};

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) { umma::tmem_ld32(addr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) { umma::tmem_ld32x16(addr, r); }

// A work item: key block [j0, end of block) of sequence b and tiles [t0, t1) of its pairs.
// What depends on the sequence alone is kept from item to item; an item costs each role a
// handful of instructions (a division proper is hundreds of cycles to a lone warp).
template <bool NARROW>
struct Work {
    static constexpr int KEYS = MK * (NARROW ? 4 : 2);
    int b = -1, end = 0, base = 0, j0 = 0, t0 = 0, t1 = 0, flats = 0, tiles = 0, per = 0, split = 0;
    // false: no key of the block is in use
    __device__ __forceinline__ bool get(const TileArgs& p, const Walk& at) {
        const AccumArgs& a = p.a;
        j0 = at.tile * KEYS;
        if (at.b != b) {
            b = at.b;
            const int live = live_rows(a.n_rows, b, a.n_q);
            base = checked_base(a.q_pos0, b, live, a.max_ctx, a.status);
            end = base + live;
            flats = live * a.heads;
            tiles = (flats + MK - 1) / MK;                     // narrow: one
            per = a.splits == 1 ? tiles : (tiles + a.splits - 1) / a.splits;
        }
        if (j0 >= end) return false;
        if (NARROW) {
            t1 = tiles;
        } else {
            split = at.part;
            t1 = min(tiles, (split + 1) * per);
            t0 = min(tiles, split * per);
            // pairs at positions before the block's first key see none of its keys
            if (j0 > base) t0 = min(t1, max(t0, (j0 - base) * a.heads / MK));
        }
        return true;
    }
};

// Slot and phase of a ring's next use.
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t size) {
        if (++slot == size) { slot = 0; phase ^= 1u; }
    }
};

// The weights of W columns of a key's lane added up: s the products, nl the pairs' -lse in log2
// units (and, MK behind, their scales), c2 the key's factor.  WHOLE: all of them count; else
// those in `see` (the others may hold anything).  Apart, and not a test per column: with the
// branches in between nothing overlapped.
template <bool KV8, bool WHOLE, bool POLY, int W>
__device__ __forceinline__ void add_weights(const uint32_t (&s)[W], const float* nl, float2 c2, uint32_t see, float2& sum0,
                                            float2& sum1) {
#pragma unroll
    for (int q = 0; q < W; q += 4) {
        const float4 n4 = *reinterpret_cast<const float4*>(nl + q);
        float2 ca = c2, cb = c2;
        if (KV8) {
            const float4 e4 = *reinterpret_cast<const float4*>(nl + MK + q);
            const float2 z = make_float2(0.f, 0.f);
            ca = fma2(c2, make_float2(e4.x, e4.y), z);
            cb = fma2(c2, make_float2(e4.z, e4.w), z);
        }
        const float2 x0 = fma2(make_float2(__uint_as_float(s[q]), __uint_as_float(s[q + 1])), ca, make_float2(n4.x, n4.y));
        const float2 x1 = fma2(make_float2(__uint_as_float(s[q + 2]), __uint_as_float(s[q + 3])), cb, make_float2(n4.z, n4.w));
        if (POLY && ((kPolyGroups >> (q / 4)) & 1u)) {
            sum0 = add_exp2_poly2(x0, sum0);
            sum1 = add_exp2_poly2(x1, sum1);
            continue;
        }
        float2 p0 = make_float2(ex2(x0.x), ex2(x0.y)), p1 = make_float2(ex2(x1.x), ex2(x1.y));
        if (!WHOLE) {
            p0.x = (see >> q) & 1u ? p0.x : 0.f;
            p0.y = (see >> (q + 1)) & 1u ? p0.y : 0.f;
            p1.x = (see >> (q + 2)) & 1u ? p1.x : 0.f;
            p1.y = (see >> (q + 3)) & 1u ? p1.y : 0.f;
        }
        sum0 = add2(sum0, p0);
        sum1 = add2(sum1, p1);
    }
}

template <int D, bool KV8, bool NARROW>
__global__ void __launch_bounds__(NT, 1) accum_tile_kernel(const __grid_constant__ CUtensorMap kmap,
                                                          const __grid_constant__ CUtensorMap qmap,
                                                          const __grid_constant__ TileArgs p) {
    using Sh = Shape<D, KV8>;
    constexpr int MT = NARROW ? 4 : 2;                         // MMAs' worth of keys per item
    extern __shared__ __align__(1024) uint8_t smem[];
    const AccumArgs& a = p.a;
    const int KS = p.k_stages, QS = p.q_slots;
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem);      // [16]
    uint64_t* k_empty = k_full + 16;                           // [16]
    uint64_t* q_full = k_empty + 16;                           // [4]
    uint64_t* q_empty = q_full + 4;                            // [4]
    uint64_t* s_full = q_empty + 4;                            // [buffer][MT]
    uint64_t* s_empty = s_full + 2 * 4;                        // [buffer][MT]
    uint64_t* nl_full = s_empty + 2 * 4;                       // [NL]
    uint64_t* nl_empty = nl_full + NL;                         // [NL]
    uint64_t* x_full = nl_empty + NL;                          // [4][2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(x_full + 8);
    volatile int& abort_flag = *reinterpret_cast<volatile int*>(tmem_slot + 1);
    float* xch = reinterpret_cast<float*>(smem + OFF_XCH);     // [4][2][MK]
    float* nls = reinterpret_cast<float*>(smem + OFF_NL);      // [NL][2][MK] lse in log2 units, Q scales
    uint8_t* qs = smem + OFF_TILES;
    uint8_t* ks = qs + QS * p.q_bytes;

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 16; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
        for (int s = 0; s < 4; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 2); }
        for (int s = 0; s < 8; ++s) { mbar_init(&s_full[s], 1); mbar_init(&s_empty[s], 4); mbar_init(&x_full[s], 4); }
        for (int s = 0; s < NL; ++s) { mbar_init(&nl_full[s], 32); mbar_init(&nl_empty[s], NARROW ? NEXP : NEXP / 2); }
        fence_mbar_init();
        abort_flag = 0;
    }
    if (warp == NEXP + 2) umma::tmem_alloc(tmem_slot, 512);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = *tmem_slot;           // S of (buffer u, keys mt): column 256 u + mt * 256 / MT
    Work<NARROW> w;
    uint32_t step = 0;                          // Q tiles so far
    bool ok = true;

    if (warp < NEXP) {
        // ---------------------------------------------------------------- exponentials
        const int quarter = warp & 3, mt = NARROW ? warp >> 2 : (warp >> 2) & 1, team = NARROW ? 0 : warp >> 3;
        const uint32_t ts = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + mt * (256 / MT);
        constexpr int W = NARROW ? 16 : 32, UN = NARROW ? 1 : 2;
        uint32_t it = 0;
        const float sc2 = a.scale * kLog2e;
        for (Walk at = p.walk.at(blockIdx.x); ok && p.walk.in(at); p.walk.next(at)) {
            if (!w.get(p, at)) continue;
            const int j = w.j0 + MK * mt + 32 * quarter + lane, n = w.t1 - w.t0;
            const int64_t key = static_cast<int64_t>(w.b) * a.cap + j;
            // the team of the last tile writes the totals
            const bool closes = NARROW || (n == 0 ? team == 0 : static_cast<int>((step + n - 1) & 1) == team);
            const bool writes = closes && j < w.end;
            float old = 0.f, ck = sc2;
            if (writes && a.splits == 1 && a.acc_in) old = a.acc_in[key];
            if (KV8 && j < w.end) ck *= __ldg(a.k_scale + key);
            // this key is seen by the pairs from here on
            const int first = max(0, min(j, w.end - 1) - w.base) * a.heads;
            float total = 0.f;
            for (int t = w.t0; t < w.t1; ++t, ++step) {
                const uint32_t u = step & 1, slot = step % NL;
                if (!NARROW && static_cast<int>(u) != team) continue;
                if (!(ok = lanes_wait(lane == 0 ? &s_full[4 * u + mt] : (lane == 1 ? &nl_full[slot] : nullptr),
                                      (lane == 0 ? step >> 1 : step / NL) & 1, &abort_flag, a.status))) break;
                umma::fence_after();
                const float2 c2 = make_float2(ck, ck);
                const int cols = min(w.flats - t * p.n_cols, p.n_cols);
                const int lo = first - t * p.n_cols;             // columns lo .. cols - 1 count
                // a chunk of columns at a time, in a loop: with a tile's 64 or 128 columns unrolled the
                // registers ran out and instructions came late
#pragma unroll UN
                for (int c0 = 0; c0 < cols; c0 += W) {
                    uint32_t s[W];
                    tmem_ld(ts + 256 * u + c0, s);
                    const bool whole = __all_sync(0xffffffffu, lo <= c0 && cols >= c0 + W);
                    const uint32_t see = whole ? 0xffffffffu : bits_below(cols - c0) & ~bits_below(lo - c0);
                    const float* nl = nls + slot * 2 * MK + c0;
                    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                    umma::tmem_ld_wait();
                    if (c0 + W >= cols) {
                        umma::fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_empty[4 * u + mt]);
                    }
                    if (whole) add_weights<KV8, true, !NARROW, W>(s, nl, c2, see, sum0, sum1);
                    else add_weights<KV8, false, false, W>(s, nl, c2, see, sum0, sum1);
                    total += (sum0.x + sum0.y) + (sum1.x + sum1.y);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&nl_empty[slot]);
            }
            if (!ok) break;
            if (!NARROW && n > 1) {
                // The other team's sums.  Four slots: S has a buffer per team and its MMAs are issued
                // in order, so that a team is at most three tiles ahead of the other.
                const uint32_t x = it % 4;
                float* slot = xch + (x * 2 + mt) * MK + 32 * quarter + lane;
                if (!closes) {
                    *slot = total;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[2 * x + mt]);
                } else {
                    if (!(ok = warp_wait(&x_full[2 * x + mt], (it / 4) & 1, &abort_flag, a.status))) break;
                    total += *slot;
                }
                ++it;
            }
            if (writes) {
                if (a.splits == 1) a.acc_out[key] = a.acc_in ? fmaf(a.decay, old, total) : total;
                else a.part[(static_cast<int64_t>(w.split) * a.batch + w.b) * a.max_ctx + j] = total;
            }
        }
    } else if (warp == NEXP) {
        // ---------------------------------------------------------------- TMA loads
        Ring kr, qr;
        uint32_t kfree = KS, qfree = QS;                       // slots never used so far need no wait
        bool split = !KV8;                                     // Q's parts are there (the keys need not wait for them)
        for (Walk at = p.walk.at(blockIdx.x); ok && p.walk.in(at); p.walk.next(at)) {
            if (!w.get(p, at) || w.t0 == w.t1) continue;
            const int krow = static_cast<int>(w.b * a.cap) + w.j0, qrow = w.b * a.n_q * a.heads;
            for (int t = w.t0; ok && t < w.t1; ++t) {
                if (t == w.t0)
                    for (int i = 0; i < MT; ++i, kr.next(KS)) {
                        if (kfree > 0) --kfree;
                        else if (!(ok = warp_wait(&k_empty[kr.slot], kr.phase ^ 1u, &abort_flag, a.status))) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&k_full[kr.slot], Sh::KTILE);
                            for (int c = 0; c < Sh::KBOXES; ++c)
                                tma_load_2d(ks + kr.slot * Sh::KTILE + c * MK * 128, &kmap, &k_full[kr.slot], c * (KV8 ? D : 64),
                                            krow + MK * i);
                        }
                    }
                if (!ok) break;
                if (qfree > 0) --qfree;
                else if (!(ok = warp_wait(&q_empty[qr.slot], qr.phase ^ 1u, &abort_flag, a.status))) break;
                if (!split) {
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                    split = true;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[qr.slot], p.n_cols * Sh::QROW);
                    for (int c = 0; c < Sh::QBOXES; ++c)
                        tma_load_2d(qs + qr.slot * p.q_bytes + c * (p.q_bytes / Sh::QBOXES), &qmap, &q_full[qr.slot],
                                    c * (KV8 ? D : 64), qrow + t * p.n_cols);
                }
                __syncwarp();
                qr.next(QS);
            }
        }
    } else if (warp == NEXP + 1) {
        // ---------------------------------------------------------------- the pairs' lse
        if (KV8) asm volatile("griddepcontrol.wait;" ::: "memory");
        for (Walk at = p.walk.at(blockIdx.x); ok && p.walk.in(at); p.walk.next(at)) {
            if (!w.get(p, at)) continue;
            const int64_t flat0 = static_cast<int64_t>(w.b) * a.n_q * a.heads;
            for (int t = w.t0; t < w.t1; ++t, ++step) {
                const uint32_t slot = step % NL;
                float v[4], e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = lane + 32 * i, f = t * p.n_cols + col;
                    const bool in = col < p.n_cols && f < w.flats;
                    v[i] = in ? -kLog2e * __ldg(a.lse + flat0 + f) : 0.f;
                    e[i] = KV8 && in ? __ldg(p.q_scale + flat0 + f) : 0.f;
                }
                if (step >= NL && !(ok = warp_wait(&nl_empty[slot], (step / NL - 1) & 1, &abort_flag, a.status))) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    nls[slot * 2 * MK + lane + 32 * i] = v[i];
                    if (KV8) nls[slot * 2 * MK + MK + lane + 32 * i] = e[i];
                }
                mbar_arrive(&nl_full[slot]);
            }
        }
    } else {
        // ---------------------------------------------------------------- MMAs
        const int odd = warp - NEXP - 2;
        Ring kr, qr;
        const uint32_t idesc = KV8 ? umma::idesc_e4m3(MK, p.n_cols) : umma::idesc_bf16(MK, p.n_cols, false, false);
        for (Walk at = p.walk.at(blockIdx.x); ok && p.walk.in(at); p.walk.next(at)) {
            if (!w.get(p, at) || w.t0 == w.t1) continue;
            const int t0 = uniform(w.t0), t1 = uniform(w.t1);
            for (int t = t0; ok && t < t1; ++t, ++step, qr.next(QS)) {
                const uint32_t u = step & 1, qslot = qr.slot;
                // this warp's 128-key tiles: slots of the ring
                Ring kx[MT / 2];
                kx[0] = kr;
                if (odd) kx[0].next(KS);
#pragma unroll
                for (int i = 1; i < MT / 2; ++i) {
                    kx[i] = kx[i - 1];
                    kx[i].next(KS);
                    kx[i].next(KS);
                }
                // lane 0: the pairs; 1, 2: S free; 3, 4: the keys
                uint64_t* bar = lane == 0 ? &q_full[qslot] : nullptr;
                uint32_t parity = qr.phase;
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    if (lane == 1 + i && step >= 2) { bar = &s_empty[4 * u + 2 * i + odd]; parity = ((step >> 1) - 1) & 1; }
                    if (lane == 3 + i && t == t0) { bar = &k_full[kx[i].slot]; parity = kx[i].phase; }
                }
                if (!(ok = lanes_wait(bar, parity, &abort_flag, a.status))) break;
                umma::fence_after();
                const uint32_t qb = smem_u32(qs) + qslot * p.q_bytes;
#pragma unroll
                for (int i = 0; i < MT / 2; ++i) {
                    const int mt = 2 * i + odd;
                    const uint32_t s = kx[i].slot;
                    const uint32_t kb = smem_u32(ks) + s * Sh::KTILE, d = tmem + 256 * u + mt * (256 / MT);
                    if (elect_one()) {
                        if (KV8) {
                            const uint64_t kd = D == 128 ? umma::sdesc_sw128(kb, 16, 1024) : umma::sdesc_sw64(kb, 512);
                            const uint64_t qh = D == 128 ? umma::sdesc_sw128(qb, 16, 1024) : umma::sdesc_sw64(qb, 512);
                            const uint64_t ql = qh + (p.q_bytes >> 5);                  // the second half of the slot
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk) umma::mma_e4m3_ss(d, kd + 2 * kk, qh + 2 * kk, idesc, kk > 0);
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk) umma::mma_e4m3_ss(d, kd + 2 * kk, ql + 2 * kk, idesc, 1u);
                        } else {
                            const uint64_t kd = umma::sdesc_sw128(kb, 16, 1024), qd = umma::sdesc_sw128(qb, 16, 1024);
                            const uint32_t qbox = p.q_bytes / Sh::QBOXES;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                umma::mma_bf16_ss(d, kd + (((kk >> 2) * (MK * 128) + (kk & 3) * 32) >> 4),
                                                  qd + (((kk >> 2) * qbox + (kk & 3) * 32) >> 4), idesc, kk > 0);
                        }
                        umma::commit(&s_full[4 * u + mt]);
                        if (t + 1 == t1) umma::commit(&k_empty[s]);
                        if (i == MT / 2 - 1) umma::commit(&q_empty[qslot]);
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) kr.next(KS);
        }
    }
    __syncwarp();
    umma::fence_before();
    __syncthreads();
    if (warp == NEXP + 2) {
        umma::fence_after();
        umma::tmem_dealloc(tmem, 512);
    }
}

// Q rows as two e4m3 numbers per element, [row][2][D], and 2^-e of each row.  16 lanes to a row.
template <int D>
__global__ void __launch_bounds__(256) accum_split_q_kernel(const __nv_bfloat16* __restrict__ q, int64_t rows,
                                                            uint8_t* __restrict__ out, float* __restrict__ scale) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");        // which wait for our end where they need it
    constexpr int PER = D / 16;                                // elements of a lane: 4 or 8
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const int l = threadIdx.x & 15;
    if (row >= rows) return;                                   // whole halves of a warp
    const uint32_t half = 0xffffu << (threadIdx.x & 16);
    float x[PER];
    uint32_t raw[PER / 2];
    if (PER == 8) {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(q + row * D) + l);
        raw[0] = r.x; raw[1] = r.y; raw[2 % (PER / 2)] = r.z; raw[3 % (PER / 2)] = r.w;
    } else {
        const uint2 r = __ldg(reinterpret_cast<const uint2*>(q + row * D) + l);
        raw[0] = r.x; raw[1] = r.y;
    }
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) {
        x[2 * i] = __uint_as_float(raw[i] << 16);
        x[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
        mx = fmaxf(mx, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(half, mx, o));
    // 2^e with mx 2^e in [128, 256); exponents kept where 2^e and 2^-e are normal numbers
    const int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 127;                   // mx in [2^ex, 2^(ex+1))
    const int e = max(-120, min(120, 7 - ex));
    const float s = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    uint32_t hi[PER / 4], lo[PER / 4];
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) {
        const float y0 = x[2 * i] * s, y1 = x[2 * i + 1] * s;
        uint16_t h, m;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y1), "f"(y0));
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(h));
        const float2 b = __half22float2(*reinterpret_cast<__half2*>(&h2));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(m) : "f"(y1 - b.y), "f"(y0 - b.x));
        if (i & 1) {
            hi[i / 2] |= static_cast<uint32_t>(h) << 16;
            lo[i / 2] |= static_cast<uint32_t>(m) << 16;
        } else {
            hi[i / 2] = h;
            lo[i / 2] = m;
        }
    }
    uint8_t* dst = out + row * 2 * D + l * PER;
    if (PER == 8) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[PER / 4 - 1]);
        *reinterpret_cast<uint2*>(dst + D) = make_uint2(lo[0], lo[PER / 4 - 1]);
    } else {
        *reinterpret_cast<uint32_t*>(dst) = hi[0];
        *reinterpret_cast<uint32_t*>(dst + D) = lo[0];
    }
    // a row with an infinity, which e4m3 has no code for: NaN for the whole row, not its largest codes
    if (l == 0) scale[row] = ex == 128 ? __int_as_float(0x7fffffff) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

template <int D, bool KV8, bool NARROW>
cudaError_t launch(TileArgs& p, const CUtensorMap& km, const CUtensorMap& qm, cudaStream_t st) {
    using Sh = Shape<D, KV8>;
    const int free_bytes = kSmem - OFF_TILES;
    p.q_bytes = (p.n_cols * Sh::QROW + 2047) / 2048 * 2048;
    p.q_slots = 2;
    p.k_stages = (free_bytes - p.q_slots * p.q_bytes) / Sh::KTILE;
    if (p.k_stages > 16) p.k_stages = 16;
    const int smem = OFF_TILES + p.q_slots * p.q_bytes + p.k_stages * Sh::KTILE;
    // The function's limit, the same in every call: another thread's call may set it before this launch.
    const cudaError_t e = cudaFuncSetAttribute(accum_tile_kernel<D, KV8, NARROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(p.walk.batch) * p.walk.tiles * p.walk.parts;
    const int grid = items < num_sms() ? static_cast<int>(items) : num_sms();
    p.walk.step = p.walk.at(grid);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = KV8 ? 1 : 0;                                // after the kernel that splits Q
    return cudaLaunchKernelEx(&cfg, accum_tile_kernel<D, KV8, NARROW>, km, qm, p);
}

template <int D, bool KV8>
cudaError_t launch_tile(const AccumArgs& a, cudaStream_t st) {
    using Sh = Shape<D, KV8>;
    TileArgs p{};
    p.a = a;
    const int64_t pairs = static_cast<int64_t>(a.n_q) * a.heads, all = a.batch * pairs;
    p.narrow = pairs <= kNarrow;
    p.n_cols = p.narrow ? static_cast<int>((pairs + 15) / 16 * 16) : MK;
    const int keys = MK * (p.narrow ? 4 : 2);
    p.walk.batch = a.batch;
    p.walk.tiles = static_cast<int>((a.max_ctx + keys - 1) / keys);
    p.walk.parts = a.splits;
    const void* q = a.q;
    if (KV8) {
        uint8_t* w = static_cast<uint8_t*>(a.split_q);
        float* scale = reinterpret_cast<float*>(w + static_cast<size_t>(all) * 2 * D);
        accum_split_q_kernel<D><<<static_cast<unsigned>((all + 15) / 16), 256, 0, st>>>(
            static_cast<const __nv_bfloat16*>(a.q), all, w, scale);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        q = w;
        p.q_scale = scale;
    }
    const uint64_t rows = static_cast<uint64_t>(a.batch) * a.cap;
    CUtensorMap km, qm;
    const CUtensorMapDataType t = KV8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int eb = KV8 ? 1 : 2;
    if (!make_tmap_2d(&km, a.k, t, eb, D, rows, Sh::ROW, Sh::KBOX / eb, MK, Sh::KBOX == 128, Sh::KBOX == 64) ||
        !make_tmap_2d(&qm, q, t, eb, KV8 ? 2 * D : D, static_cast<uint64_t>(all), Sh::QROW, Sh::KBOX / eb,
                      static_cast<uint32_t>(p.n_cols), Sh::KBOX == 128, Sh::KBOX == 64))
        return cudaErrorInvalidValue;
    return p.narrow ? launch<D, KV8, true>(p, km, qm, st) : launch<D, KV8, false>(p, km, qm, st);
}

}  // namespace

cudaError_t launch_accum_tile(const AccumArgs& a, cudaStream_t st) {
    if (a.kv_dtype == HS2_E4M3) return a.head_dim == 128 ? launch_tile<128, true>(a, st) : launch_tile<64, true>(a, st);
    return a.head_dim == 128 ? launch_tile<128, false>(a, st) : launch_tile<64, false>(a, st);
}

}  // namespace hs2
