// window_tile.cu -- attention over a sliding window and the first tokens (sinks) for chunks
// of query rows, on tcgen05.
//
// The query at position p attends to rows j <= p with j > p - W or j < S.  All heads share
// the one K/V head, so 256 consecutive (row, head) pairs of a sequence are stacked in the
// MMA's M dimension as two halves of 128, and both halves consume every K and V tile that
// the CTA loads.  The keys that any of the 256 pairs sees form one list (KeyList); it is cut
// into tiles of 128, the last one as short as the list allows (a multiple of 16), so that a
// window of 128 costs 160 columns and not 256.
//
// Per half and tile:  S = Q K^T into tensor memory; one thread per pair reads its row of S
// into registers, masks it, and forms P = 2^(S sc2 - m), which goes back over S as packed
// bf16 and is the A operand of O += P V.  m is a reference that trails the running maximum by
// at most 2^8: it moves, and O is rescaled in place, only when the maximum rises by more than
// 8 in log2 units, which after a row's first tile is rare; sums and O are fp32 and P keeps
// bf16's relative rounding of 2^-8 whatever its magnitude, so nothing is lost by it.
//
// S(i + 1) of a half is issued right behind PV(i) of the same half by the same thread: the
// tensor pipe executes one thread's MMAs in issue order, so P(i) has been read before S(i + 1)
// overwrites it, and S(i + 1) being complete means that O holds PV(i).  While one half's
// threads form P the tensor cores work for the other half.  P goes out in two parts, so that PV
// runs while the rest of the exponentials is formed (8192 rows, window 4096: 353 us in two parts,
// 415 in one, 390 in four).
//
// Work items (sequence, 256 pairs, part of the keys) are dealt to one persistent CTA per SM,
// and the roles run ahead of one another across items: the next item's Q, K and V are loaded
// while this one is computed, and its first S is formed while this one's O is written out.
//
// Roles (384 threads): warps 0-3 and 4-7 the softmax and the output of halves 0 and 1, warp 8
// the loads, warps 9 and 10 the MMAs of halves 0 and 1 (a step of waits, descriptors and
// commits is some 500 cycles of latency to its warp; in one warp the halves held each other
// up).  The softmax threads hold a row of S in registers (208 each, taken from the others).
// Every wait is bounded; a wait that gives up flags the status word and makes all roles leave
// their loops.
//
// e4m3 caches: the codes of the rows that the call attends to are first widened to bf16
// (exact) in the workspace; the rows' scales multiply S and P in fp32.
//
// Measured (16 heads of 128, bf16, replayed from a graph on the same inputs): 8192 rows with a
// window of 4096 353 us (780 TFLOP/s; 4700 cycles a tile of 128 keys, of which the MMAs are 2048,
// the exponentials' unit 1800 and the softmax threads' instructions 3200: the chain S, softmax, PV
// of a half bounds it), 4 x 8192 rows with a window of 128 117 us.  As calls among others on
// changing inputs: 355 and 119.
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "tile_sync.cuh"
#include "window_keys.cuh"

namespace hs2 {
namespace {

constexpr int KT = 128;                         // keys per tile
constexpr int MH = 128;                         // pairs per half
constexpr int PART = 64, PARTS = KT / PART;     // keys of P handed over at a time
constexpr int NT = 384;
constexpr int NSOFT = 8;                        // softmax warps; then one for loads and two for MMAs
constexpr int STAGES = 3;                       // K and V tiles in flight, K(t) at 2t, V(t) at 2t + 1
constexpr int QSLOTS = 3;                       // halves of Q held: an item's two and the next one's first
constexpr int SC_SLOTS = 4;                     // tiles whose scales are held (at most 3 are live)
constexpr int ST_BYTES = 32 * 64;               // a warp's O on its way out: 32 rows of 32 columns
constexpr float kLag = 8.f;                     // log2 units the reference may trail the maximum by
// tensor memory: S and P of half h at column 128 h, O at 256 + 128 h
constexpr uint32_t kOcol = 256;

template <int D>
struct Shape {
    static constexpr int ROW = D * 2;                          // bytes of a bf16 row
    static constexpr int BOXES = D / 64;                       // 64-column swizzled boxes per tile
    static constexpr int BOX = KT * 128, QBOX = MH * 128;      // bytes of a box
    static constexpr int TILE = BOXES * BOX, QTILE = BOXES * QBOX;
    static constexpr int BARS = 320;                          // barriers, the tensor-memory base, the abort flag
    // all of it dynamic, so that the tiles start 1024-byte aligned without padding
    static constexpr int OFF_KV = QSLOTS * QTILE, OFF_OUT = OFF_KV + STAGES * TILE, OFF_RING = OFF_OUT + NSOFT * ST_BYTES,
                         OFF_BARS = OFF_RING + SC_SLOTS * 2 * KT * 4, SMEM = OFF_BARS + BARS;
    static_assert(SMEM <= 232448, "shared memory of a CTA");
};

struct TileArgs {
    WindowArgs w;
    WalkPlan walk;                              // (sequence, 256 pairs, part of the keys)
    FastDiv heads;
    int64_t cap;                                // rows per sequence of the maps' K and V
    int s16;                                    // e4m3: widened sink rows per sequence
    uint32_t* status;
};

// First widened cache row of a sequence: its first row's window start, or 0 where the sinks
// reach it (then no sink lies before the window's range of any row).
__device__ __forceinline__ int widened_lo(int base, int window, int sinks) {
    const int lo = max(0, base - window + 1);
    return sinks >= lo ? 0 : lo;
}

// One work item: which pairs and which tiles of their key list.  Consecutive items of a CTA
// mostly belong to one sequence, whose position and length are kept from item to item.
struct Work {
    int b, f0, f_last, base, live, t0, t1, split, shift;       // shift: map row of cache row r in the window part
    KeyList kl;
    __device__ __forceinline__ Work() : b(-1), kl(0, 0, 1, 0) {}
    // false: no pairs in use.  t0 == t1: no keys in this part.
    __device__ __forceinline__ bool get(const TileArgs& a, const Walk& at) {
        const WindowArgs& w = a.w;
        split = at.part;
        f0 = at.tile * 2 * MH;
        if (at.b != b) {
            b = at.b;
            live = live_rows(w.n_rows, b, w.n_q);
            base = checked_base(w.q_pos0, b, live, w.max_ctx, a.status);
        }
        if (f0 >= live * w.heads) return false;
        f_last = min(f0 + 2 * MH - 1, live * w.heads - 1);
        kl = KeyList(base + a.heads.div(f0), base + a.heads.div(f_last), w.window, w.sinks);
        const int n = (kl.total + KT - 1) / KT, per = w.splits == 1 ? n : (n + w.splits - 1) / w.splits;
        t0 = min(n, split * per);
        t1 = min(n, t0 + per);
        shift = w.kv_dtype == HS2_E4M3 ? a.s16 - widened_lo(base, w.window, w.sinks) : 0;
        return true;
    }
    __device__ __forceinline__ int halves() const { return f_last - f0 >= MH ? 2 : 1; }
    // columns of tile t, to a multiple of 16
    __device__ __forceinline__ int cols(int t) const { return min(KT, (kl.total - t * KT + 15) & ~15); }
};

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    umma::fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
// Descriptors of a tile's first K step (K-major with its 64-column boxes, MN-major), of which
// the steps differ in the address field alone.
__device__ __forceinline__ uint64_t kmajor(uint32_t base) { return umma::sdesc_sw128(base, 16, 1024); }
__device__ __forceinline__ uint64_t mnmajor(uint32_t base) { return umma::sdesc_sw128(base, KT * 128, 1024); }
__device__ __forceinline__ uint64_t kstep(uint64_t d, int kk) { return d + (((kk >> 2) * (KT * 128) + (kk & 3) * 32) >> 4); }
__device__ __forceinline__ uint64_t mnstep(uint64_t d, int kk) { return d + kk * (2048 >> 4); }

template <int D, bool KV8>
__global__ void __launch_bounds__(NT, 1) window_tile_kernel(const __grid_constant__ CUtensorMap qmap,
                                                           const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap,
                                                           const __grid_constant__ CUtensorMap kmap16,
                                                           const __grid_constant__ CUtensorMap vmap16,
                                                           const __grid_constant__ TileArgs a) {
    using Sh = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem;                                        // Q slots
    uint8_t* st = smem + Sh::OFF_KV;                           // K and V stages
    float* ring = reinterpret_cast<float*>(smem + Sh::OFF_RING);          // [SC_SLOTS][2][KT] scales (e4m3)
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Sh::OFF_BARS);
    uint64_t* q_empty = q_full + QSLOTS;
    uint64_t* kv_full = q_empty + QSLOTS;
    uint64_t* kv_empty = kv_full + STAGES;
    uint64_t* s_full = kv_empty + STAGES;                      // [half]
    uint64_t* p_full = s_full + 2;                             // [half][part]
    uint64_t* o_full = p_full + 2 * PARTS;                     // [half]
    uint64_t* sc_full = o_full + 2;                            // [SC_SLOTS]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_full + SC_SLOTS);
    volatile int& abort_flag = *reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * QSLOTS + 2 * STAGES + 4 + 2 * PARTS + SC_SLOTS) * 8 + 8 <= Sh::BARS, "barriers fit");

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int h = 0; h < 2; ++h) {
            mbar_init(&s_full[h], 1); mbar_init(&o_full[h], 1);
            for (int i = 0; i < PARTS; ++i) mbar_init(&p_full[PARTS * h + i], 4);
        }
        for (int s = 0; s < QSLOTS; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1); }
        for (int s = 0; s < STAGES; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 2); }
        for (int s = 0; s < SC_SLOTS; ++s) mbar_init(&sc_full[s], 32);
        fence_mbar_init();
        abort_flag = 0;
    }
    if (warp == NSOFT + 1) umma::tmem_alloc(tmem_slot, 512);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < NSOFT) {
        // ---------------------------------------------------------------- softmax, output
        regs_inc<208>();
        const int h = warp >> 2, quarter = warp & 3, m_row = quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + KT * h, to = tmem + lanes + kOcol + 128 * h;
        uint8_t* sw = smem + Sh::OFF_OUT + warp * ST_BYTES;
        const float sc2 = a.w.scale * kLog2e;
        uint32_t gt = 0, ht = 0, hi = 0;        // tiles so far; tiles and items of this half
        bool ok = true;
        Work w;
        for (Walk pos = a.walk.at(blockIdx.x); ok && a.walk.in(pos); a.walk.next(pos)) {
            if (!w.get(a, pos)) continue;
            const int f = w.f0 + MH * h + m_row;
            const int64_t flat = static_cast<int64_t>(w.b) * a.w.n_q * a.w.heads + f;
            const int64_t at = static_cast<int64_t>(w.split) * a.w.batch * a.w.n_q * a.w.heads + flat;
            if (w.t0 == w.t1) {                                 // only of split keys: an empty part
                if (f <= w.f_last) a.w.part_ml[at] = make_float2(-INFINITY, 0.f);
                continue;
            }
            if (h >= w.halves()) { gt += w.t1 - w.t0; continue; }
            // this pair sees list entries [lo_u, hi_u] and those below s_u
            int lo_u = 0, hi_u = -1, s_u = 0;
            if (f <= w.f_last) {
                const int p = w.base + a.heads.div(f);
                lo_u = max(p - a.w.window + 1 - w.kl.lo, 0) + w.kl.s_pad;
                hi_u = p - w.kl.lo + w.kl.s_pad;
                s_u = w.kl.lo > 0 ? w.kl.s_eff : min(a.w.sinks, p + 1);
            }
            float m = -INFINITY, l = 0.f;
            for (int t = w.t0; t < w.t1; ++t, ++gt, ++ht) {
                if (!(ok = warp_wait(&s_full[h], ht & 1, &abort_flag, a.status))) break;
                if (KV8 && !(ok = warp_wait(&sc_full[gt % SC_SLOTS], (gt / SC_SLOTS) & 1, &abort_flag, a.status))) break;
                umma::fence_after();
                const int u0 = t * KT, cols = w.cols(t), nc = (cols + 31) >> 5;
                const float* ksc = ring + (gt % SC_SLOTS) * 2 * KT;
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < nc) umma::tmem_ld32(ts + 32 * i, s[i]);
                umma::tmem_ld_wait();
                const bool masked = __any_sync(0xffffffffu, u0 < lo_u || u0 + KT - 1 > hi_u);
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < nc) {
                        if (KV8) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 k4 = *reinterpret_cast<const float4*>(ksc + 32 * i + j);
                                s[i][j] = __float_as_uint(__uint_as_float(s[i][j]) * k4.x);
                                s[i][j + 1] = __float_as_uint(__uint_as_float(s[i][j + 1]) * k4.y);
                                s[i][j + 2] = __float_as_uint(__uint_as_float(s[i][j + 2]) * k4.z);
                                s[i][j + 3] = __float_as_uint(__uint_as_float(s[i][j + 3]) * k4.w);
                            }
                        }
                        if (masked) {
                            const int cb = u0 + 32 * i;
                            const uint32_t see = (bits_below(hi_u - cb + 1) & ~bits_below(lo_u - cb)) | bits_below(s_u - cb);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((see >> j) & 1u)) s[i][j] = 0xff800000u;              // -inf
                        }
                        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            m0 = max3(m0, __uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1]));
                            m1 = max3(m1, __uint_as_float(s[i][j + 2]), __uint_as_float(s[i][j + 3]));
                        }
                        mx = max3(mx, m0, m1);
                    }
                mx *= sc2;
                if (m == -INFINITY && mx > m) m = mx;           // nothing summed yet: l and O's row are zero
                const bool move = mx > m + kLag;
                if (__any_sync(0xffffffffu, move)) {
                    const float r = move ? ex2(m - mx) : 1.f;
                    l *= r;
                    if (move) m = mx;
                    if (t > w.t0) {
#pragma unroll 1
                        for (int d = 0; d < D; d += 16) {
                            uint32_t o[16];
                            umma::tmem_ld32x16(to + d, o);
                            umma::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * r);
                            umma::tmem_st32x16(to + d, o);
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.f : m;
                const float2 s2 = make_float2(sc2, sc2), nm = make_float2(-off, -off);
                float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < nc) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float2 x0 = fma2(make_float2(__uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1])), s2, nm);
                            const float2 x1 = fma2(make_float2(__uint_as_float(s[i][j + 2]), __uint_as_float(s[i][j + 3])), s2, nm);
                            float2 p0 = make_float2(ex2(x0.x), ex2(x0.y)), p1 = make_float2(ex2(x1.x), ex2(x1.y));
                            sum0 = add2(sum0, p0);
                            sum1 = add2(sum1, p1);
                            // rounded to bf16 for the MMA (2^-8 relative), next to e4m3 rows times the value's scale
                            if (KV8) {
                                const float4 v4 = *reinterpret_cast<const float4*>(ksc + KT + 32 * i + j);
                                p0.x *= v4.x; p0.y *= v4.y; p1.x *= v4.z; p1.y *= v4.w;
                            }
                            pk[j / 2] = pack_bf16(p0.x, p0.y);
                            pk[j / 2 + 1] = pack_bf16(p1.x, p1.y);
                        }
                        umma::tmem_st32x16(ts + 16 * i, pk);
                    }
                    if (i == 0) {
                        // V rows of entries that hold no key may hold anything, and 0 * NaN would poison O
                        if (!KV8 && (u0 + KT > w.kl.total || (u0 < w.kl.s_pad && w.kl.s_eff < w.kl.s_pad))) {
                            const uint32_t vi = 2 * gt + 1;
                            if (m_row < cols && w.kl.row(u0 + m_row) < 0 &&
                                wait_or_abort(&kv_full[vi % STAGES], (vi / STAGES) & 1, &abort_flag, a.status)) {
                                uint8_t* vrow = st + (vi % STAGES) * Sh::TILE + m_row * 128;
#pragma unroll
                                for (int c = 0; c < Sh::BOXES * 8; ++c)
                                    *reinterpret_cast<uint4*>(vrow + (c >> 3) * Sh::BOX + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                                umma::fence_proxy_async();
                            }
                            __syncwarp();
                        }
                    }
                    if (i % (PART / 32) == PART / 32 - 1) {
                        umma::tmem_st_wait();
                        warp_arrive(&p_full[PARTS * h + i / (PART / 32)]);
                    }
                }
                l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
            }
            if (!ok || !(ok = warp_wait(&o_full[h], hi & 1, &abort_flag, a.status))) break;
            ++hi;
            umma::fence_after();
            const float inv = a.w.splits == 1 ? 1.f / l : 1.f;
#pragma unroll
            for (int d = 0; d < D; d += 32) {
                uint32_t o[32];
                umma::tmem_ld32(to + d, o);
                umma::tmem_ld_wait();
                if (a.w.splits > 1) {
                    if (f <= w.f_last) {
                        uint4* dst = reinterpret_cast<uint4*>(a.w.part_o + at * D + d);
#pragma unroll
                        for (int j = 0; j < 8; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                    continue;
                }
                // 32 rows x 64 bytes through shared memory (16-byte chunk j of row r at j ^ (r / 2) % 4),
                // so that each store instruction writes whole sectors
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(sw + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(pack_bf16(__uint_as_float(o[8 * j]) * inv, __uint_as_float(o[8 * j + 1]) * inv),
                                   pack_bf16(__uint_as_float(o[8 * j + 2]) * inv, __uint_as_float(o[8 * j + 3]) * inv),
                                   pack_bf16(__uint_as_float(o[8 * j + 4]) * inv, __uint_as_float(o[8 * j + 5]) * inv),
                                   pack_bf16(__uint_as_float(o[8 * j + 6]) * inv, __uint_as_float(o[8 * j + 7]) * inv));
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 8 * j + (lane >> 2), ch = lane & 3;
                    const uint4 x = *reinterpret_cast<const uint4*>(sw + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
                    if (f - lane + r <= w.f_last)
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.w.o) + (flat - lane + r) * D + d + 8 * ch) = x;
                }
            }
            if (f <= w.f_last) {
                if (a.w.splits > 1) a.w.part_ml[at] = make_float2(m, l);
                else if (a.w.lse) a.w.lse[flat] = (m + log2f(l)) * kLn2;
            }
        }
    } else {
        regs_dec<80>();
        if (warp == NSOFT && (KV8 || lane == 0)) {
            // ------------------------------------------------------------ loads
            uint32_t n = 0, gt = 0, qn = 0;                       // stage uses, tiles, Q slot uses
            bool ok = true;
            auto load_q = [&](const Work& w, int h) {
                const uint32_t s = qn % QSLOTS;
                bool go = true;
                if (lane == 0) {
                    if (qn >= QSLOTS) go = wait_or_abort(&q_empty[s], (qn / QSLOTS - 1) & 1, &abort_flag, a.status);
                    if (go) {
                        const int row = w.b * a.w.n_q * a.w.heads + w.f0 + MH * h;
                        mbar_arrive_expect_tx(&q_full[s], Sh::QTILE);
                        for (int c = 0; c < Sh::BOXES; ++c)
                            tma_load_2d(qs + s * Sh::QTILE + c * Sh::QBOX, &qmap, &q_full[s], 64 * c, row);
                    }
                }
                ++qn;
                return KV8 ? __shfl_sync(0xffffffffu, static_cast<int>(go), 0) != 0 : go;
            };
            Work w;
            for (Walk pos = a.walk.at(blockIdx.x); ok && a.walk.in(pos); a.walk.next(pos)) {
                if (!w.get(a, pos) || w.t0 == w.t1) continue;
                const int nh = w.halves();
                const int krow = static_cast<int>(w.b * a.cap);
                if (!(ok = load_q(w, 0))) break;
                for (int t = w.t0; ok && t < w.t1; ++t, ++gt) {
                    const int u0 = t * KT, groups = w.cols(t) >> 4;
                    for (int kv = 0; kv < 2; ++kv, ++n) {
                        const int s = n % STAGES;
                        if (lane == 0 && n >= STAGES)
                            ok = wait_or_abort(&kv_empty[s], ((n / STAGES) - 1) & 1, &abort_flag, a.status);
                        if (KV8) ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        if (lane == 0) {
                            uint8_t* dst = st + s * Sh::TILE;
                            if (u0 >= w.kl.s_pad && groups == KT / 16) {        // one box
                                const CUtensorMap* map = kv ? &vmap : &kmap;
                                const int row = krow + w.kl.lo + w.shift + u0 - w.kl.s_pad;
                                mbar_arrive_expect_tx(&kv_full[s], Sh::TILE);
                                for (int c = 0; c < Sh::BOXES; ++c)
                                    tma_load_2d(dst + c * Sh::BOX, map, &kv_full[s], 64 * c, row);
                            } else {                                             // boxes of 16 rows
                                const CUtensorMap* map = kv ? &vmap16 : &kmap16;
                                mbar_arrive_expect_tx(&kv_full[s], groups * 16 * Sh::ROW);
                                for (int g = 0; g < groups; ++g) {
                                    const int u = u0 + 16 * g;
                                    const int row = krow + (u < w.kl.s_pad ? u : w.kl.lo + w.shift + u - w.kl.s_pad);
                                    for (int c = 0; c < Sh::BOXES; ++c)
                                        tma_load_2d(dst + c * Sh::BOX + g * 2048, map, &kv_full[s], 64 * c, row);
                                }
                            }
                        }
                        if (kv == 0) {
                            if (KV8) {          // the tile's 128 K and V scales, each lane's copies arriving as they land
                                float* slot = ring + (gt % SC_SLOTS) * 2 * KT;
                                const int64_t seq0 = static_cast<int64_t>(w.b) * a.w.cap;
#pragma unroll
                                for (int j = 0; j < KT / 32; ++j) {
                                    const int key = w.kl.row(u0 + lane + 32 * j);
                                    const int64_t src = seq0 + max(key, 0);
                                    cp_async4_zfill(slot + lane + 32 * j, a.w.k_scale + src, key >= 0);
                                    cp_async4_zfill(slot + KT + lane + 32 * j, a.w.v_scale + src, key >= 0);
                                }
                                cp_async_arrive_noinc(&sc_full[gt % SC_SLOTS]);
                            }
                            if (t == w.t0 && nh == 2 && !(ok = load_q(w, 1))) break;
                        }
                    }
                }
            }
            if (KV8) asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == NSOFT + 1 || warp == NSOFT + 2) {
            // ------------------------------------------------------------ MMAs of a half
            // The whole warp walks, one elected lane issues.  S runs a tile ahead of PV, which
            // keeps what it needs of the tile before.
            const int h = warp - NSOFT - 1;
            constexpr uint32_t idesc_o = umma::idesc_bf16(128, D, false, true);
            const uint64_t qd = kmajor(smem_u32(qs)), kd = kmajor(smem_u32(st)), vd = mnmajor(smem_u32(st));
            const uint32_t tp = tmem + KT * h, to = tmem + kOcol + 128 * h;
            Work w;
            Walk pos = a.walk.at(blockIdx.x);
            int t = 0, total = 0, t0 = 0, t1 = 0, nh = 0;
            auto seek = [&]() {
                nh = 0;
                for (; a.walk.in(pos); a.walk.next(pos))
                    if (w.get(a, pos) && w.t0 < w.t1) {
                        t = t0 = uniform(w.t0); t1 = uniform(w.t1); total = uniform(w.kl.total); nh = uniform(w.halves());
                        return;
                    }
            };
            uint32_t gs = 0, gp = 0, qn = 0, ht = 0;              // tiles of S and of PV, Q slots, PV tiles of this half
            bool ok = true;
            auto issue_s = [&]() {
                const uint32_t s = (2 * gs) % STAGES;
                if (!(ok = warp_wait(&kv_full[s], (2 * gs / STAGES) & 1, &abort_flag, a.status))) return;
                if (h >= nh) {                                    // the other half alone reads this stage
                    if (lane == 0) mbar_arrive(&kv_empty[s]);
                    return;
                }
                const uint32_t qslot = (qn + h) % QSLOTS;
                if (t == t0 && !(ok = warp_wait(&q_full[qslot], ((qn + h) / QSLOTS) & 1, &abort_flag, a.status))) return;
                umma::fence_after();
                const uint32_t idesc_s = umma::idesc_bf16(128, min(KT, (total - t * KT + 15) & ~15), false, false);
                const uint64_t qh = qd + qslot * (Sh::QTILE >> 4), kb = kd + s * (Sh::TILE >> 4);
                const bool last = t + 1 == t1;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma::mma_bf16_ss(tp, kstep(qh, kk), kstep(kb, kk), idesc_s, kk > 0);
                    umma::commit(&s_full[h]);
                    umma::commit(&kv_empty[s]);
                    if (last) umma::commit(&q_empty[qslot]);
                }
                __syncwarp();
            };
            seek();
            if (nh > 0) issue_s();
            while (ok && nh > 0) {
                const int steps = min(KT / 16, (total - t * KT + 15) >> 4);
                const bool mine = h < nh, last = t + 1 == t1;
                const uint32_t old = t > t0 ? 1u : 0u, s = (2 * gp + 1) % STAGES;
                const uint64_t vb = vd + s * (Sh::TILE >> 4);
                ++gs;
                if (++t == t1) { qn += nh; a.walk.next(pos); seek(); }
                if (!(ok = warp_wait(&kv_full[s], ((2 * gp + 1) / STAGES) & 1, &abort_flag, a.status))) break;
                if (mine) {
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        if (!(ok = warp_wait(&p_full[PARTS * h + part], ht & 1, &abort_flag, a.status))) break;
                        umma::fence_after();
                        const int k0 = part * (PART / 16), k1 = min(steps, k0 + PART / 16);
                        if (elect_one()) {
                            if (k1 == k0 + PART / 16) {
#pragma unroll
                                for (int kk = 0; kk < PART / 16; ++kk)
                                    umma::mma_bf16_ts(to, tp + 8 * (k0 + kk), mnstep(vb, k0 + kk), idesc_o, k0 + kk > 0 ? 1u : old);
                            } else {
                                for (int kk = k0; kk < k1; ++kk)
                                    umma::mma_bf16_ts(to, tp + 8 * kk, mnstep(vb, kk), idesc_o, kk > 0 ? 1u : old);
                            }
                            if (part == PARTS - 1) {
                                umma::commit(&kv_empty[s]);
                                if (last) umma::commit(&o_full[h]);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    ++ht;
                } else if (lane == 0) {
                    mbar_arrive(&kv_empty[s]);
                }
                if (nh > 0) issue_s();
                ++gp;
            }
        }
    }
    __syncwarp();
    umma::fence_before();
    __syncthreads();
    if (warp == NSOFT + 1) {
        umma::fence_after();
        umma::tmem_dealloc(tmem, 512);
    }
}

// The rows that the call attends to, codes widened to bf16 (exact), per sequence: the sinks at
// rows 0 .. s16 - 1, then the cache rows from the first window's start to the last position,
// and 16 zero rows (the end of a list is read to a multiple of 16).  8 codes of K and V per
// thread and step.
template <int D>
__global__ void __launch_bounds__(256) window_widen_kernel(WindowArgs a, int blocks, int s16, int64_t rows,
                                                           __nv_bfloat16* __restrict__ kw, __nv_bfloat16* __restrict__ vw) {
    constexpr int PER = D / 8;
    const int b = blockIdx.x / blocks;
    const int live = live_rows(a.n_rows, b, a.n_q);
    if (live == 0) return;
    const int base = checked_base(a.q_pos0, b, live, a.max_ctx, a.status);
    const int lo = widened_lo(base, a.window, a.sinks), last = base + live - 1;
    const int64_t used = min(rows, static_cast<int64_t>(s16) + last - lo + 1 + 16);
    const int64_t step = static_cast<int64_t>(blocks) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x - b * blocks) * blockDim.x + threadIdx.x; i < used * PER; i += step) {
        const int64_t r = i / PER;
        const int c = static_cast<int>(i - r * PER);
        int key = -1;
        if (r < s16) {
            if (r < a.sinks && r <= last) key = static_cast<int>(r);
        } else if (r - s16 <= last - lo) {
            key = lo + static_cast<int>(r - s16);
        }
        uint4 ko = make_uint4(0, 0, 0, 0), vo = ko;
        if (key >= 0) {
            const int64_t src = (static_cast<int64_t>(b) * a.cap + key) * D + c * 8;
            const uint2 kc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.k) + src));
            const uint2 vc = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v) + src));
            ko = make_uint4(e4m3x2_to_bf16x2(kc.x & 0xffff), e4m3x2_to_bf16x2(kc.x >> 16),
                            e4m3x2_to_bf16x2(kc.y & 0xffff), e4m3x2_to_bf16x2(kc.y >> 16));
            vo = make_uint4(e4m3x2_to_bf16x2(vc.x & 0xffff), e4m3x2_to_bf16x2(vc.x >> 16),
                            e4m3x2_to_bf16x2(vc.y & 0xffff), e4m3x2_to_bf16x2(vc.y >> 16));
        }
        const int64_t dst = static_cast<int64_t>(b) * rows + r;
        reinterpret_cast<uint4*>(kw + dst * D)[c] = ko;
        reinterpret_cast<uint4*>(vw + dst * D)[c] = vo;
    }
}

template <int D, bool KV8>
cudaError_t launch(const WindowArgs& w, cudaStream_t st) {
    using Sh = Shape<D>;
    TileArgs a{};
    a.w = w;
    a.status = w.status;
    a.heads = FastDiv(static_cast<uint32_t>(w.heads));
    a.walk.batch = w.batch;
    a.walk.tiles = static_cast<int>((static_cast<int64_t>(w.n_q) * w.heads + 2 * MH - 1) / (2 * MH));
    a.walk.parts = w.splits;
    const int64_t items = static_cast<int64_t>(a.walk.batch) * a.walk.tiles * a.walk.parts;
    const int grid = items < num_sms() ? static_cast<int>(items) : num_sms();
    a.walk.step = a.walk.at(grid);
    a.cap = w.cap;
    const void* k = w.k;
    const void* v = w.v;
    if (KV8) {
        a.s16 = window_sink_rows(w.sinks, w.max_ctx);
        a.cap = w.wide_rows;
        __nv_bfloat16* kw = static_cast<__nv_bfloat16*>(w.wide);
        __nv_bfloat16* vw = kw + static_cast<size_t>(w.batch) * w.wide_rows * D;
        const int64_t work = (w.wide_rows * (D / 8) + 255) / 256;
        const int64_t most = 8 * static_cast<int64_t>(num_sms()) / w.batch + 1;
        const int blocks = static_cast<int>(work < most ? work : most);
        window_widen_kernel<D><<<static_cast<unsigned>(blocks) * w.batch, 256, 0, st>>>(w, blocks, a.s16, w.wide_rows, kw, vw);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        k = kw;
        v = vw;
    }
    const uint64_t pairs = static_cast<uint64_t>(w.batch) * w.n_q * w.heads, rows = static_cast<uint64_t>(w.batch) * a.cap;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap qm, km, vm, km16, vm16;
    if (!make_tmap_2d(&qm, w.q, bf, 2, D, pairs, Sh::ROW, 64, MH, true) ||
        !make_tmap_2d(&km, k, bf, 2, D, rows, Sh::ROW, 64, KT, true) ||
        !make_tmap_2d(&vm, v, bf, 2, D, rows, Sh::ROW, 64, KT, true) ||
        !make_tmap_2d(&km16, k, bf, 2, D, rows, Sh::ROW, 64, 16, true) ||
        !make_tmap_2d(&vm16, v, bf, 2, D, rows, Sh::ROW, 64, 16, true))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(window_tile_kernel<D, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::SMEM);
    if (e != cudaSuccess) return e;
    window_tile_kernel<D, KV8><<<static_cast<unsigned>(grid), NT, Sh::SMEM, st>>>(qm, km, vm, km16, vm16, a);
    return cudaGetLastError();
}

}  // namespace

int window_sink_rows(int sinks, int64_t max_ctx) {
    const int64_t s = sinks < max_ctx ? sinks : max_ctx;
    return static_cast<int>((s + kSinkPad - 1) / kSinkPad * kSinkPad);
}

int64_t window_wide_rows(int n_q, int window, int sinks, int64_t max_ctx) {
    int64_t span = static_cast<int64_t>(window) + n_q + sinks;
    if (span > max_ctx) span = max_ctx;
    return window_sink_rows(sinks, max_ctx) + span + 16;
}

cudaError_t launch_window_tile(const WindowArgs& a, cudaStream_t st) {
    if (a.kv_dtype == HS2_E4M3) return a.head_dim == 128 ? launch<128, true>(a, st) : launch<64, true>(a, st);
    return a.head_dim == 128 ? launch<128, false>(a, st) : launch<64, false>(a, st);
}

}  // namespace hs2
