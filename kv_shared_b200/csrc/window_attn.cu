// window_attn.cu -- attention over a sliding window and the first tokens (sinks): the
// kernels for single tokens and small chunks (bf16 and e4m3 caches), the fp32 kernel, and
// the join of split keys.
//
// The query at position p attends to rows j <= p with j > p - W or j < S.  All heads share
// the one K/V head, so (row, head) pairs are stacked: 16 consecutive pairs of a sequence
// share every key that any of their rows attends to.
//
// Single tokens are bound by reading K and V once.  Each warp takes steps of 16 keys from its
// own ring of asynchronous copies in shared memory (no barrier but its own in the loop; with
// one step ahead in registers a step took the memory's latency, 2.9 TB/s), and keeps the step
// itself in registers.  For S = Q K^T thread (g, t) of a warp holds 16-byte chunks t, t + 4, ..
// of key g's row, which is a permutation of the contraction index that Q's fragments follow;
// for O += P V it holds chunk g of keys 2t, 2t + 1, 2t + 8, 2t + 9, whose dims become the MMA's
// n index (a permutation of the output columns, undone on the way out).  Rows are stored with
// their chunks shifted so that neither read meets a bank twice.  The warps' running (max, sum,
// O) are joined in shared memory; with few rows and many keys the keys are cut over CTAs as
// well and a second launch joins the parts in a fixed order.  Measured (16 heads of 128; times in
// this file are replayed from a graph on the same inputs): 32 tokens, window 128, 5.8 us; 4 tokens,
// window 32768, e4m3, 15.1 us (2.3 TB/s).  As calls among others on changing inputs: 8.0 and 18.4.
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "tile_sync.cuh"
#include "window_keys.cuh"

namespace hs2 {
namespace {

constexpr int NW = 8;                            // warps per CTA
constexpr int STEP = 16;                         // keys per warp step
constexpr float kLag = 4.f;                      // log2 units: weights stay below 2^4, f16's products far from its end
constexpr int kMinSplitKeys = 512;               // keys per CTA below which a split costs more than it saves
constexpr int F_QT = 8;                          // fp32: threads that share a few pairs
constexpr int F_ROWS = 32;                       // (row, head) pairs per CTA
constexpr int F_KEYS = 32;                       // keys per tile
constexpr int kMinSplitKeysF32 = 32;
constexpr int kMinSplitKeysTile = 256;

template <int D, bool KV8>
struct Frag {
    static constexpr int ROW = D * (KV8 ? 1 : 2);        // bytes of a cache row
    static constexpr int KC = ROW / 64;                  // 16-byte K chunks per thread and 8 keys
    static constexpr int VB = ROW / 8;                   // V bytes per thread and key: 8, 16 or 32
    static constexpr int VW = VB / 4;                    // in 32-bit words
    static constexpr int CPR = ROW / 16;                 // chunks of a row
    static constexpr int PLANE = STEP * ROW;             // K or V of a step
    static constexpr int STAGE = 2 * PLANE + (KV8 ? 2 * STEP * 4 : 0);      // K, V, their scales
    // as many stages as shared memory has room for, up to 6
    static constexpr int STAGES = 200 * 1024 / NW / STAGE < 6 ? 200 * 1024 / NW / STAGE : 6;
    uint4 k[2][KC];                                      // [8-key half][chunk]
    uint32_t v[4][VW];                                   // [key 2t, 2t+1, 2t+8, 2t+9][words]
    float ks[4], vs[4];                                  // scales of the same keys (e4m3)

    // where chunk c of row r lies in its plane: K is read by rows (neighbours' chunks t), V by
    // every second row (one chunk)
    static __device__ __forceinline__ int k_at(int r, int c) {
        return r * ROW + ((CPR >= 8 ? (c & ~7) | ((c + 4 * (r & 1)) & 7) : c) << 4);
    }
    static __device__ __forceinline__ int v_at(int r, int c) {
        return r * ROW + ((CPR >= 8 ? (c & ~7) | ((c + 2 * ((r >> 1) & 3)) & 7) : (c + ((r >> 1) & 3)) & 3) << 4);
    }
    // the copies of keys u0 .. u0 + 15 of the list into a stage (whole warp); rows that hold no
    // key become zeros
    static __device__ __forceinline__ void copy(uint8_t* st, const WindowArgs& a, int64_t seq0, const KeyList& kl, int u0,
                                                int end, int lane) {
        constexpr int RPC = 32 / CPR < 1 ? 1 : 32 / CPR;         // rows per 32 chunks
        const int c = lane % CPR;
#pragma unroll
        for (int r0 = 0; r0 < STEP; r0 += RPC) {
            const int r = r0 + lane / CPR, u = u0 + r;
            const int key = u < end ? kl.row(u) : -1;
            const int64_t src = (seq0 + max(key, 0)) * ROW + c * 16;
            cp_async16_zfill(st + k_at(r, c), static_cast<const uint8_t*>(a.k) + src, key >= 0);
            cp_async16_zfill(st + PLANE + v_at(r, c), static_cast<const uint8_t*>(a.v) + src, key >= 0);
        }
        if (KV8) {
            const int r = lane & 15, u = u0 + r;
            const int key = u < end ? kl.row(u) : -1;
            cp_async4_zfill(st + 2 * PLANE + lane * 4, (lane < 16 ? a.k_scale : a.v_scale) + seq0 + max(key, 0), key >= 0);
        }
    }
    __device__ __forceinline__ void load(const uint8_t* st, int g, int t) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < KC; ++c) k[h][c] = *reinterpret_cast<const uint4*>(st + k_at(8 * h + g, t + 4 * c));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * (i >> 1) + 2 * t + (i & 1);
            if (VB == 8) {
                const uint2 x = *reinterpret_cast<const uint2*>(st + PLANE + v_at(r, g >> 1) + 8 * (g & 1));
                v[i][0] = x.x; v[i][1] = x.y;
            } else {
#pragma unroll
                for (int c = 0; c < VB / 16; ++c) {
                    const uint4 x = *reinterpret_cast<const uint4*>(st + PLANE + v_at(r, g + 8 * c));
                    v[i][4 * c % VW] = x.x; v[i][(4 * c + 1) % VW] = x.y;
                    v[i][(4 * c + 2) % VW] = x.z; v[i][(4 * c + 3) % VW] = x.w;
                }
            }
            if (KV8) {
                ks[i] = *reinterpret_cast<const float*>(st + 2 * PLANE + 4 * r);
                vs[i] = *reinterpret_cast<const float*>(st + 2 * PLANE + 4 * (16 + r));
            }
        }
    }
};

// First of the 16 consecutive output dims of thread t that n-tiles 8c .. 8c+7 hold: dims
// +0..7 in the fragment's even column, +8..15 in the odd one (e4m3 rows of 128: 32 dims
// from 16 n-tiles, 16 per column).
template <int D, bool KV8>
__device__ __forceinline__ int out_dim(int nt, int col, int t) {
    return Frag<D, KV8>::VB == 16 && KV8 ? 16 * (2 * t + col) + nt : (nt >> 3) * 64 + 8 * (2 * t + col) + (nt & 7);
}

template <int D, bool KV8>
__global__ void __launch_bounds__(NW * 32, 1) window_rows_kernel(WindowArgs a, FastDiv heads, FastDiv tiles, FastDiv parts) {
    using F = Frag<D, KV8>;
    constexpr int KS = D / 16;                   // k-steps of S
    constexpr int NT = D / 8;                    // n-tiles of O
    constexpr int LDO = D + 4;                   // row pitch of the join
    // the warps' rings; at the end [NW][16][LDO] O, then [NW][16] max, [NW][16] sum
    extern __shared__ float sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int b = tiles.div(blockIdx.x), f0 = (blockIdx.x - b * static_cast<int>(tiles.d)) * 16;
    const int split = blockIdx.y;
    const int live = live_rows(a.n_rows, b, a.n_q);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");         // the join may be set up; it waits for our end
    if (f0 >= live * a.heads) return;
    const int base = checked_base(a.q_pos0, b, live, a.max_ctx, a.status);
    const int f_last = min(f0 + 15, live * a.heads - 1);
    const KeyList kl(base + heads.div(f0), base + heads.div(f_last), a.window, a.sinks);
    const int chunk = a.splits == 1 ? kl.total : (parts.div(kl.total + a.splits - 1) + STEP - 1) / STEP * STEP;
    const int begin = min(kl.total, split * chunk), end = min(kl.total, begin + chunk);
    const int64_t seq0 = static_cast<int64_t>(b) * a.cap;
    const int64_t flat0 = static_cast<int64_t>(b) * a.n_q * a.heads;

    uint8_t* ring = reinterpret_cast<uint8_t*>(sm) + warp * (F::STAGES * F::STAGE);
    int u0 = begin + warp * STEP;
#pragma unroll
    for (int i = 0; i < F::STAGES - 1; ++i) {
        if (u0 + i * NW * STEP < end) F::copy(ring + i * F::STAGE, a, seq0, kl, u0 + i * NW * STEP, end, lane);
        cp_async_commit();
    }
    // Q fragments of pairs g and g + 8 in the keys' order of dims, and the pairs' positions
    uint32_t qa[KS][4];
    int pos[2];
    float mag = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int fr = f0 + g + 8 * r;
        pos[r] = fr <= f_last ? base + heads.div(fr) : -1;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (flat0 + fr) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d = KV8 ? 16 * (t + 4 * (ks >> 2)) + 4 * (ks & 3) : 8 * (t + 4 * (ks >> 1)) + 4 * (ks & 1);
            const uint2 x = fr <= f_last ? __ldg(reinterpret_cast<const uint2*>(q + d)) : make_uint2(0, 0);
            qa[ks][r] = x.x;
            qa[ks][2 + r] = x.y;
        }
    }
    float sc2 = a.scale * kLog2e;
    if (KV8) {
        // Q as f16 next to the codes' f16: times a power of two that brings its largest magnitude
        // to [2^13, 2^14); what falls below f16's range then is 2^-38 of that
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mag = fmaxf(mag, fmaxf(fabsf(__uint_as_float(qa[ks][i] << 16)), fabsf(__uint_as_float(qa[ks][i] & 0xffff0000u))));
        mag = warp_max(mag);
        const int e = max(-120, min(120, 13 - (static_cast<int>(__float_as_uint(mag) >> 23) - 127)));
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qa[ks][i] = pack_f16(__uint_as_float(qa[ks][i] << 16) * up, __uint_as_float(qa[ks][i] & 0xffff0000u) * up);
        sc2 *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    }

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // list entries open_lo .. open_hi - 1 hold keys that all sixteen pairs see (where sinks lie
    // inside the window's range, that range alone)
    const int p_lo = base + heads.div(f0), p_hi = base + heads.div(f_last);
    const int open_lo = f_last - f0 < 15 ? end : max(kl.s_pad, kl.s_pad + p_hi - a.window + 1 - kl.lo);
    const int open_hi = min(end, kl.s_pad + p_lo - kl.lo + 1);

    for (int stage = 0; u0 < end; u0 += NW * STEP) {
        const int un = u0 + (F::STAGES - 1) * NW * STEP;
        int free = stage + F::STAGES - 1;                        // the stage read last
        if (free >= F::STAGES) free -= F::STAGES;
        if (un < end) F::copy(ring + free * F::STAGE, a, seq0, kl, un, end, lane);
        cp_async_commit();
        cp_async_wait<F::STAGES - 1>();
        __syncwarp();
        F f;
        f.load(ring + stage * F::STAGE, g, t);
        __syncwarp();                                            // before the next turn's copies into it
        if (++stage == F::STAGES) stage = 0;
        float s[2][4], lift[4];
        if (KV8) {
            // The value's scale belongs to its weight: weights are kept relative to the largest
            // weight times scale, so that in f16 they are at most 2^kLag and what f16 drops is
            // 2^-25 of it.
#pragma unroll
            for (int i = 0; i < 4; ++i) lift[i] = fminf(fmaxf(__log2f(f.vs[i]), -60.f), 60.f);
        }
        float mn[2] = {m[0], m[1]};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[h][j] = 0.f;
#pragma unroll
            for (int c = 0; c < F::KC; ++c) {
                const uint32_t w[4] = {f.k[h][c].x, f.k[h][c].y, f.k[h][c].z, f.k[h][c].w};
                if (KV8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16x2x2(w[i], b0, b1);
                        mma_f16(s[h], qa[4 * c + i], b0, b1);
                    }
                } else {
                    mma_bf16(s[h], qa[2 * c], w[0], w[1]);
                    mma_bf16(s[h], qa[2 * c + 1], w[2], w[3]);
                }
            }
        }
        float kf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kf[i] = KV8 ? f.ks[i] * sc2 : sc2;
        // logits in log2 units, hidden keys at -inf; most steps hide none
        const bool whole = u0 >= open_lo && u0 + STEP <= open_hi;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[h][j] *= kf[2 * h + (j & 1)];
        if (!whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = u0 + 8 * h + 2 * t + (j & 1);
                    const int key = u < end ? kl.row(u) : -1;
                    if (!window_sees(key, pos[j >> 1], a.window, a.sinks)) s[h][j] = -INFINITY;
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mn[j >> 1] = fmaxf(mn[j >> 1], KV8 ? s[h][j] + lift[2 * h + (j & 1)] : s[h][j]);
        // the reference may trail the maximum by kLag: O is rescaled now and then, not every step
        bool rose = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 1));
            mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 2));
            if (!(mn[r] > m[r] + kLag)) mn[r] = m[r] == -INFINITY ? mn[r] : m[r];
            rose |= mn[r] > m[r];
        }
        if (__any_sync(0xffffffffu, rose)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float c = m[r] == -INFINITY ? 1.f : ex2(m[r] - mn[r]);       // from -inf: l and O are zero
                l[r] *= c;
                m[r] = mn[r];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    o[i][2 * r] *= c;
                    o[i][2 * r + 1] *= c;
                }
            }
        }
        uint32_t pa[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float off = m[r] == -INFINITY ? 0.f : m[r];
                const float p0 = ex2(s[h][2 * r] - off), p1 = ex2(s[h][2 * r + 1] - off);
                l[r] += p0 + p1;
                // the MMA's operand type: a rounding of at most 2^-11 relative (f16), 2^-8 (bf16)
                pa[2 * h + r] = KV8 ? pack_f16(p0 * f.vs[2 * h], p1 * f.vs[2 * h + 1]) : pack_bf16(p0, p1);
            }
#pragma unroll
        for (int w = 0; w < F::VW; ++w) {
            if (KV8) {
                // bytes of keys (2t, 2t + 1) side by side, then widened
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t sel = q ? 0x7362u : 0x5140u;
                    uint32_t a0, a1, b0, b1;
                    e4m3x4_to_f16x2x2(prmt(f.v[0][w], f.v[1][w], sel), a0, a1);
                    e4m3x4_to_f16x2x2(prmt(f.v[2][w], f.v[3][w], sel), b0, b1);
                    mma_f16(o[(4 * w + 2 * q) % NT], pa, a0, b0);
                    mma_f16(o[(4 * w + 2 * q + 1) % NT], pa, a1, b1);
                }
            } else {
                mma_bf16(o[(2 * w) % NT], pa, prmt(f.v[0][w], f.v[1][w], 0x5410u), prmt(f.v[2][w], f.v[3][w], 0x5410u));
                mma_bf16(o[(2 * w + 1) % NT], pa, prmt(f.v[0][w], f.v[1][w], 0x7632u),
                         prmt(f.v[2][w], f.v[3][w], 0x7632u));
            }
        }
    }

    // join the warps: pairs' maxima and sums, then O scaled to the common maximum, in the rings'
    // memory.  A thread's dims come in runs of four.
    cp_async_wait<0>();
    __syncthreads();
    float* so = sm;
    float* s_m = sm + NW * 16 * LDO;
    float* s_l = s_m + NW * 16;
    const int active = min(NW, (end - begin + STEP - 1) / STEP);           // warps with keys
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t == 0) {
            // a NaN query leaves no maximum, but a sum that is to be joined: any number serves as its reference
            s_m[warp * 16 + g + 8 * r] = l[r] != l[r] ? 0.f : m[r];
            s_l[warp * 16 + g + 8 * r] = l[r];
        }
    }
    if (warp < active) {
#pragma unroll
        for (int i = 0; i < NT; i += 4)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4*>(so + (warp * 16 + g + 8 * (j >> 1)) * LDO + out_dim<D, KV8>(i, j & 1, t)) =
                    make_float4(o[i][j], o[i + 1][j], o[i + 2][j], o[i + 3][j]);
    }
    __syncthreads();
    // NW * 32 / 16 threads to a pair, each with the same share of its dims
    constexpr int TPP = NW * 2, PER = D / TPP;                             // 8 (4) dims
    const int r = threadIdx.x / TPP, d = threadIdx.x % TPP * PER;
    if (f0 + r > f_last) return;
    float mw[NW], mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        mw[w] = w < active ? s_m[w * 16 + r] : -INFINITY;
        mx = fmaxf(mx, mw[w]);
    }
    float sum = 0.f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        if (mw[w] != -INFINITY) {
            const float c = ex2(mw[w] - mx);
            sum = fmaf(c, s_l[w * 16 + r], sum);
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(so + (w * 16 + r) * LDO + d + i);
                acc[i] = fmaf(c, x.x, acc[i]); acc[i + 1] = fmaf(c, x.y, acc[i + 1]);
                acc[i + 2] = fmaf(c, x.z, acc[i + 2]); acc[i + 3] = fmaf(c, x.w, acc[i + 3]);
            }
        }
    const int64_t flat = flat0 + f0 + r;
    if (a.splits == 1) {
        const float inv = 1.f / sum;
#pragma unroll
        for (int i = 0; i < PER; i += 4)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + flat * D + d + i) =
                make_uint2(pack_bf16(acc[i] * inv, acc[i + 1] * inv), pack_bf16(acc[i + 2] * inv, acc[i + 3] * inv));
        if (a.lse && d == 0) a.lse[flat] = (mx + log2f(sum)) * kLn2;
    } else {
        const int64_t at = static_cast<int64_t>(split) * a.batch * a.n_q * a.heads + flat;
#pragma unroll
        for (int i = 0; i < PER; i += 4)
            *reinterpret_cast<float4*>(a.part_o + at * D + d + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        if (d == 0) a.part_ml[at] = make_float2(mx, sum);
    }
}

// fp32: 32 pairs x 32 keys per tile on the CUDA cores (a bf16 or tf32 product would lose what
// the fp32 caches are there for).  Thread (rp, qt) of 32 / RP x 8 has pairs RP rp .. RP rp + RP - 1;
// keys qt + 8 i of S, dims 4 (qt + 8 j) of O, two fp32 FMAs to an instruction.  RP = 4 makes 8 loads
// of 16 bytes from shared memory to 64 FMAs and is bound by them and by latency: 2 x 1023 rows of 8
// heads of 64, window 128, 25.7 us (RP = 2, 12 to 64: 31.4).  RP = 2 has twice the warps, for calls
// that leave each SM a CTA at most and are bound by a tile's latency alone, some 2 us: one row of 16
// heads of 128, window 4096, 4 sinks, 13.9 us (RP = 4: 18.5; parts of 256 keys: 37.7); without sinks
// 11.0, for the keys then divide into 128 parts of a tile, where otherwise parts round up to two
// tiles and half of them have no keys.
template <int D, int RP>
__global__ void __launch_bounds__(F_ROWS / RP * F_QT) window_f32_kernel(WindowArgs a) {
    constexpr int NT = F_ROWS / RP * F_QT;
    constexpr int LDQ = D + 4;                   // row pitch: rows of a quarter-warp on distinct banks
    constexpr int LDP = F_KEYS + 4;
    constexpr int NC = D / (4 * F_QT);           // float4 chunks of O per thread and pair
    constexpr int KPT = F_KEYS / F_QT;           // keys of S per thread and pair
    extern __shared__ float4 sm4[];
    float* sq = reinterpret_cast<float*>(sm4);   // [F_ROWS][LDQ]
    float* sp = sq + F_ROWS * LDQ;               // [F_ROWS][LDP]
    float* kv = sp + F_ROWS * LDP;               // [2] K [F_KEYS][LDQ], V [F_KEYS][D]: a tile ahead
    const int tid = threadIdx.x, rp = tid / F_QT, qt = tid % F_QT;
    const int tiles = (a.n_q * a.heads + F_ROWS - 1) / F_ROWS;
    const int b = blockIdx.x / tiles, f0 = (blockIdx.x - b * tiles) * F_ROWS;
    const int live = live_rows(a.n_rows, b, a.n_q);
    if (f0 >= live * a.heads) return;
    const int base = checked_base(a.q_pos0, b, live, a.max_ctx, a.status);
    const int f_last = min(f0 + F_ROWS - 1, live * a.heads - 1);
    const KeyList kl(base + f0 / a.heads, base + f_last / a.heads, a.window, a.sinks);
    const int chunk = ((kl.total + a.splits - 1) / a.splits + F_KEYS - 1) / F_KEYS * F_KEYS;
    const int begin = min(kl.total, static_cast<int>(blockIdx.y) * chunk), end = min(kl.total, begin + chunk);
    const int64_t seq0 = static_cast<int64_t>(b) * a.cap;
    const int64_t flat0 = static_cast<int64_t>(b) * a.n_q * a.heads;
    const float sc2 = a.scale * kLog2e;

    for (int i = tid; i < F_ROWS * D / 4; i += NT) {
        const int r = i / (D / 4), c = i - r * (D / 4);
        const float4 x = f0 + r <= f_last ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (flat0 + f0 + r) * D) + c)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(sq + r * LDQ + 4 * c) = x;
    }
    int pos[RP];
    float m[RP], l[RP];
    float4 o[RP][NC];
#pragma unroll
    for (int r = 0; r < RP; ++r) {
        const int f = f0 + RP * rp + r;
        pos[r] = f <= f_last ? base + f / a.heads : -1;
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto copy = [&](int u0, int buf) {
        float* sk = kv + buf * F_KEYS * (LDQ + D);
        float* sv = sk + F_KEYS * LDQ;
#pragma unroll
        for (int i = tid; i < F_KEYS * D / 4; i += NT) {
            const int r = i / (D / 4), c = i - r * (D / 4);
            const int key = u0 + r < end ? kl.row(u0 + r) : -1;
            const int64_t src = (seq0 + max(key, 0)) * D + 4 * c;
            cp_async16_zfill(sk + r * LDQ + 4 * c, static_cast<const float*>(a.k) + src, key >= 0);
            cp_async16_zfill(sv + r * D + 4 * c, static_cast<const float*>(a.v) + src, key >= 0);
        }
    };
    if (begin < end) copy(begin, 0);
    cp_async_commit();
    int buf = 0;
    for (int u0 = begin; u0 < end; u0 += F_KEYS, buf ^= 1) {
        if (u0 + F_KEYS < end) copy(u0 + F_KEYS, buf ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const float* sk = kv + buf * F_KEYS * (LDQ + D);
        const float* sv = sk + F_KEYS * LDQ;
        float2 d[RP][KPT];                     // sums over the even and the odd dims
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int i = 0; i < KPT; ++i) d[r][i] = make_float2(0.f, 0.f);
#pragma unroll (RP == 2 ? 8 : 4)
        for (int c = 0; c < D / 4; ++c) {
            float4 x[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) x[r] = *reinterpret_cast<const float4*>(sq + (RP * rp + r) * LDQ + 4 * c);
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(sk + (qt + F_QT * i) * LDQ + 4 * c);
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    d[r][i] = fma2(make_float2(x[r].x, x[r].y), make_float2(y.x, y.y),
                                   fma2(make_float2(x[r].z, x[r].w), make_float2(y.z, y.w), d[r][i]));
            }
        }
        float s[RP][KPT];
#pragma unroll
        for (int r = 0; r < RP; ++r)
#pragma unroll
            for (int i = 0; i < KPT; ++i) s[r][i] = d[r][i].x + d[r][i].y;
        int key[KPT];
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const int u = u0 + qt + F_QT * i;
            key[i] = u < end ? kl.row(u) : -1;
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                s[r][i] = window_sees(key[i], pos[r], a.window, a.sinks) ? s[r][i] * sc2 : -INFINITY;
                mx = fmaxf(mx, s[r][i]);
            }
#pragma unroll
            for (int o1 = 1; o1 < F_QT; o1 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o1));
            const float mn = fmaxf(m[r], mx);
            const float c = mn == -INFINITY ? 1.f : exp2f(m[r] - mn), off = mn == -INFINITY ? 0.f : mn;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                const float p = exp2f(s[r][i] - off);
                sum += p;
                sp[(RP * rp + r) * LDP + qt + F_QT * i] = p;
            }
            l[r] = fmaf(l[r], c, sum);
            m[r] = mn;
#pragma unroll
            for (int j = 0; j < NC; ++j) { o[r][j].x *= c; o[r][j].y *= c; o[r][j].z *= c; o[r][j].w *= c; }
        }
        __syncwarp();                            // a pair's weights come from its F_QT neighbouring threads
#pragma unroll 4
        for (int k = 0; k < F_KEYS; k += 4) {
            float4 w[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) w[r] = *reinterpret_cast<const float4*>(sp + (RP * rp + r) * LDP + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    const float4 y = *reinterpret_cast<const float4*>(sv + (k + i) * D + 4 * (qt + F_QT * j));
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const float p = i == 0 ? w[r].x : i == 1 ? w[r].y : i == 2 ? w[r].z : w[r].w;
                        const float2 lo = fma2(make_float2(p, p), make_float2(y.x, y.y), make_float2(o[r][j].x, o[r][j].y));
                        const float2 hi = fma2(make_float2(p, p), make_float2(y.z, y.w), make_float2(o[r][j].z, o[r][j].w));
                        o[r][j] = make_float4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
        }
        __syncthreads();                         // the tile may be overwritten
    }
#pragma unroll
    for (int r = 0; r < RP; ++r) {
#pragma unroll
        for (int o1 = 1; o1 < F_QT; o1 <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o1);
        const int f = f0 + RP * rp + r;
        if (f > f_last) continue;
        const int64_t flat = flat0 + f;
        const int64_t at = static_cast<int64_t>(blockIdx.y) * a.batch * a.n_q * a.heads + flat;
        const float inv = a.splits == 1 ? 1.f / l[r] : 1.f;
        float* dst = a.splits == 1 ? static_cast<float*>(a.o) + flat * D : a.part_o + at * D;
#pragma unroll
        for (int j = 0; j < NC; ++j)
            *reinterpret_cast<float4*>(dst + 4 * (qt + F_QT * j)) =
                make_float4(o[r][j].x * inv, o[r][j].y * inv, o[r][j].z * inv, o[r][j].w * inv);
        if (qt == 0) {
            if (a.splits > 1) a.part_ml[at] = make_float2(m[r], l[r]);
            else if (a.lse) a.lse[flat] = (m[r] + log2f(l[r])) * kLn2;
        }
    }
}

// Joins the parts of a pair: D / 4 threads with four dims each and JOIN_Y of them to a pair,
// which take the parts in turn; their sums are added in order.
constexpr int JOIN_Y = 8;
template <typename T, int D>
__global__ void __launch_bounds__(D / 4 * JOIN_Y) window_join_kernel(WindowArgs a, FastDiv rows) {
    // Launched early: the parts are there from here on.  Before any return, or a call of no rows
    // would be over before the kernel ahead of it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t all = static_cast<int64_t>(a.batch) * a.n_q * a.heads;
    const int64_t flat = blockIdx.x;
    const int b = rows.div(static_cast<int>(flat));              // rows.d: pairs per sequence
    if (flat - static_cast<int64_t>(b) * rows.d >= static_cast<int64_t>(live_rows(a.n_rows, b, a.n_q)) * a.heads) return;
    const int d = threadIdx.x * 4, y = threadIdx.y;
    float mx = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int AHEAD = 5;                                     // parts in flight per thread
    for (int s0 = y; s0 < a.splits; s0 += JOIN_Y * AHEAD) {
        float2 ml[AHEAD];
        float4 x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int s = s0 + i * JOIN_Y;
            ml[i] = s < a.splits ? a.part_ml[s * all + flat] : make_float2(-INFINITY, 0.f);
            x[i] = s < a.splits ? *reinterpret_cast<const float4*>(a.part_o + (s * all + flat) * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (ml[i].y == 0.f) continue;                        // a part without keys may have left no O (NaN: a NaN query's)
            const float mn = fmaxf(mx, ml[i].x), c0 = exp2f(mx - mn), c1 = exp2f(ml[i].x - mn);
            sum = fmaf(sum, c0, c1 * ml[i].y);
            acc.x = fmaf(acc.x, c0, c1 * x[i].x); acc.y = fmaf(acc.y, c0, c1 * x[i].y);
            acc.z = fmaf(acc.z, c0, c1 * x[i].z); acc.w = fmaf(acc.w, c0, c1 * x[i].w);
            mx = mn;
        }
    }
    __shared__ float4 s_o[JOIN_Y][D / 4];
    __shared__ float2 s_ml[JOIN_Y];
    s_o[y][threadIdx.x] = acc;
    if (threadIdx.x == 0) s_ml[y] = make_float2(mx, sum);
    __syncthreads();
    if (y > 0) return;
    mx = s_ml[0].x;
#pragma unroll
    for (int i = 1; i < JOIN_Y; ++i) mx = fmaxf(mx, s_ml[i].x);
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < JOIN_Y; ++i) {
        const float c = s_ml[i].y == 0.f ? 0.f : exp2f(s_ml[i].x - mx);
        const float4 x = s_o[i][threadIdx.x];
        sum = fmaf(c, s_ml[i].y, sum);
        acc.x = fmaf(c, x.x, acc.x); acc.y = fmaf(c, x.y, acc.y);
        acc.z = fmaf(c, x.z, acc.z); acc.w = fmaf(c, x.w, acc.w);
    }
    const float inv = 1.f / sum;
    T* dst = static_cast<T*>(a.o) + flat * D + d;
    dst[0] = static_cast<T>(acc.x * inv); dst[1] = static_cast<T>(acc.y * inv);
    dst[2] = static_cast<T>(acc.z * inv); dst[3] = static_cast<T>(acc.w * inv);
    if (a.lse && threadIdx.x == 0) a.lse[flat] = (mx + log2f(sum)) * kLn2;
}

template <int D, bool KV8>
cudaError_t launch_rows(const WindowArgs& a, cudaStream_t st) {
    constexpr int join = (NW * 16 * (D + 4) + 2 * NW * 16) * 4, rings = NW * Frag<D, KV8>::STAGES * Frag<D, KV8>::STAGE;
    constexpr int smem = join > rings ? join : rings;
    const cudaError_t e = cudaFuncSetAttribute(window_rows_kernel<D, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (static_cast<unsigned>(a.n_q) * a.heads + 15) / 16;
    window_rows_kernel<D, KV8><<<dim3(tiles * a.batch, a.splits), NW * 32, smem, st>>>(a, FastDiv(a.heads), FastDiv(tiles), FastDiv(a.splits));
    return cudaGetLastError();
}

template <int D, int RP>
cudaError_t launch_f32(const WindowArgs& a, unsigned tiles, cudaStream_t st) {
    constexpr int smem = (F_ROWS * (D + 4) + F_ROWS * (F_KEYS + 4) + 2 * F_KEYS * (2 * D + 4)) * 4;
    const cudaError_t e = cudaFuncSetAttribute(window_f32_kernel<D, RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    window_f32_kernel<D, RP><<<dim3(tiles * a.batch, a.splits), F_ROWS / RP * F_QT, smem, st>>>(a);
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_f32(const WindowArgs& a, cudaStream_t st) {
    const unsigned tiles = (static_cast<unsigned>(a.n_q) * a.heads + F_ROWS - 1) / F_ROWS;
    return static_cast<int64_t>(tiles) * a.batch * a.splits > num_sms() ? launch_f32<D, 4>(a, tiles, st)
                                                                        : launch_f32<D, 2>(a, tiles, st);
}

template <typename T, int D>
cudaError_t launch_join(const WindowArgs& a, cudaStream_t st) {
    const int64_t all = static_cast<int64_t>(a.batch) * a.n_q * a.heads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(all));
    cfg.blockDim = dim3(D / 4, JOIN_Y);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, window_join_kernel<T, D>, a, FastDiv(static_cast<uint32_t>(a.n_q) * a.heads));
}

}  // namespace

namespace {

// One kernel's launch: (row, head) pairs and keys per CTA, parts the keys are cut into, rounds of
// CTAs on the SMs.
struct Shape {
    int64_t tiles, keys, parts, rounds;
};
Shape shape(int batch, int64_t pairs, int heads, int window, int sinks, int64_t max_ctx, int rows, int per_sm, int min_keys) {
    Shape s;
    s.tiles = (pairs + rows - 1) / rows * batch;
    // keys of a tile: its rows' windows and the sinks, at most the whole context
    s.keys = static_cast<int64_t>(window) + rows / heads + sinks + kSinkPad;
    if (s.keys > max_ctx + kSinkPad) s.keys = max_ctx + kSinkPad;
    // parts: as many as fill the SMs once, each with enough keys to be worth the join
    s.parts = num_sms() * per_sm / s.tiles;
    if (s.parts > s.keys / min_keys) s.parts = s.keys / min_keys;
    if (s.parts < 1) s.parts = 1;
    s.rounds = (s.tiles * s.parts + num_sms() * per_sm - 1) / (num_sms() * per_sm);
    return s;
}

}  // namespace

WindowPlan plan_window(int batch, int n_q, int heads, int kv_dtype, int window, int sinks, int64_t max_ctx) {
    const int64_t pairs = static_cast<int64_t>(n_q) * heads;
    WindowPlan p{};
    if (kv_dtype == HS2_F32) {
        p.splits = static_cast<int>(shape(batch, pairs, heads, window, sinks, max_ctx, F_ROWS, 2, kMinSplitKeysF32).parts);
        return p;
    }
    const Shape r = shape(batch, pairs, heads, window, sinks, max_ctx, 16, 1, kMinSplitKeys);
    const Shape t = shape(batch, pairs, heads, window, sinks, max_ctx, 256, 1, kMinSplitKeysTile);
    // The tcgen05 kernel is the faster one per key but slow to start and to join, so the small
    // calls are left to the other.  Both estimated, in tenths of a microsecond, from what they
    // measured (bf16, 16 heads; rows kernel against tile kernel): 64 rows, window 128, 5.9 us
    // against 11.6; 8 x 64 rows: 19.4 against 11.8; 4 x 64 rows, window 1000: 23.6 against 38.5;
    // 256 rows, window 4000: 71 against 41; 8192 rows: 1350 against 120.
    const int64_t cost_r = 40 + r.rounds * (9 * ((r.keys / r.parts + 127) / 128) + 20) + (r.parts > 1 ? 50 : 0);
    const int64_t cost_t = 80 + t.rounds * 35 * ((t.keys / t.parts + 127) / 128) +
                           (t.parts > 1 ? 50 + batch * pairs * t.parts / 500 : 0);
    p.tile = pairs > 16 && cost_t < cost_r;
    p.splits = static_cast<int>(p.tile ? t.parts : r.parts);
    if (p.tile && kv_dtype == HS2_E4M3) p.wide_rows = window_wide_rows(n_q, window, sinks, max_ctx);
    return p;
}

size_t window_wide_bytes(int batch, int head_dim, const WindowPlan& p) {
    return static_cast<size_t>(2) * batch * p.wide_rows * head_dim * 2;
}

size_t window_ws_bytes(int batch, int n_q, int heads, int head_dim, const WindowPlan& p) {
    const size_t parts = p.splits <= 1 ? 0 : static_cast<size_t>(batch) * n_q * heads * p.splits * (head_dim * sizeof(float) + sizeof(float2));
    return window_wide_bytes(batch, head_dim, p) + parts;
}

cudaError_t launch_window(const WindowArgs& a, cudaStream_t st) {
    cudaError_t e;
    const bool d128 = a.head_dim == 128;
    if (a.tile) e = launch_window_tile(a, st);
    else if (a.kv_dtype == HS2_F32) e = d128 ? launch_f32<128>(a, st) : launch_f32<64>(a, st);
    else if (a.kv_dtype == HS2_BF16) e = d128 ? launch_rows<128, false>(a, st) : launch_rows<64, false>(a, st);
    else e = d128 ? launch_rows<128, true>(a, st) : launch_rows<64, true>(a, st);
    if (e != cudaSuccess || a.splits == 1) return e;
    if (a.kv_dtype == HS2_F32) return d128 ? launch_join<float, 128>(a, st) : launch_join<float, 64>(a, st);
    return d128 ? launch_join<__nv_bfloat16, 128>(a, st) : launch_join<__nv_bfloat16, 64>(a, st);
}

}  // namespace hs2
