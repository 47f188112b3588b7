// window_attn.cu -- attention over a sliding window and the first tokens (sinks): the
// kernels for single tokens and small chunks (bf16 and e4m3 caches), the fp32 kernel, and
// the join of split keys.
//
// The query at position p attends to rows j <= p with j > p - W or j < S.  All heads share
// the one K/V head, so (row, head) pairs are stacked: 16 consecutive pairs of a sequence
// share every key that any of their rows attends to.
//
// Single tokens are bound by reading K and V once.  A warp takes 16 keys per step and keeps
// the whole step in registers: keys and values come by 16-byte loads straight into the
// fragments of m16n8k16 MMAs, no shared memory and no barrier in the loop.  For S = Q K^T
// thread (g, t) of a warp holds chunks t, t + 4, .. of key g's row, which is a permutation of
// the contraction index that Q's fragments follow; for O += P V it holds chunk g of keys 2t,
// 2t + 1, 2t + 8, 2t + 9, whose dims become the MMA's n index (a permutation of the output
// columns, undone on the way out).  The next step's keys are loaded as soon as S is formed
// and its values as soon as they are used, so 4 to 8 KB per warp are always in flight.  The
// warps' running (max, sum, O) are joined in shared memory; with few rows and many keys the
// keys are cut over CTAs as well and a second launch joins the parts in a fixed order.
#include "common.cuh"
#include "internal.h"
#include "window_keys.cuh"

namespace hs2 {
namespace {

constexpr int NW = 8;                            // warps per CTA
constexpr int STEP = 16;                         // keys per warp step
constexpr int kMinSplitKeys = 512;               // keys per CTA below which a split costs more than it saves
constexpr int F_ROWS = 64;                       // fp32: (row, head) pairs per CTA
constexpr int F_KEYS = 32;                       // fp32: keys per tile
constexpr int kMinSplitKeysF32 = 256;
constexpr int64_t kTilePairs = 129;               // (row, head) pairs per sequence from which the tcgen05 kernel is taken

// Four e4m3 codes -> two bf16 pairs, exact.
__device__ __forceinline__ void codes_to_bf16(uint32_t v, uint32_t& lo, uint32_t& hi) {
    lo = e4m3x2_to_bf16x2(static_cast<uint16_t>(v & 0xffffu));
    hi = e4m3x2_to_bf16x2(static_cast<uint16_t>(v >> 16));
}

template <int D, bool KV8>
struct Frag {
    static constexpr int ROW = D * (KV8 ? 1 : 2);        // bytes of a cache row
    static constexpr int KC = ROW / 64;                  // 16-byte K chunks per thread and 8 keys
    static constexpr int VB = ROW / 8;                   // V bytes per thread and key: 8, 16 or 32
    static constexpr int VW = VB / 4;                    // in 32-bit words
    uint4 k[2][KC];                                      // [8-key half][chunk]
    uint32_t v[4][VW];                                   // [key 2t, 2t+1, 2t+8, 2t+9][words]
    float ks[4], vs[4];                                  // scales of the same keys (e4m3)
};

template <int D, bool KV8>
__device__ __forceinline__ void load_k(Frag<D, KV8>& f, const WindowArgs& a, int64_t seq0, const KeyList& kl, int u0,
                                       int end, int g, int t) {
    using F = Frag<D, KV8>;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int u = u0 + 8 * h + g;
        const int key = u < end ? kl.row(u) : -1;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.k) + (seq0 + key) * F::ROW);
#pragma unroll
        for (int c = 0; c < F::KC; ++c)
            f.k[h][c] = key >= 0 ? __ldg(src + t + 4 * c) : make_uint4(0, 0, 0, 0);
    }
    if (KV8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = u0 + 8 * (i >> 1) + 2 * t + (i & 1);
            const int key = u < end ? kl.row(u) : -1;
            f.ks[i] = key >= 0 ? __ldg(a.k_scale + seq0 + key) : 0.f;
        }
    }
}

template <int D, bool KV8>
__device__ __forceinline__ void load_v(Frag<D, KV8>& f, const WindowArgs& a, int64_t seq0, const KeyList& kl, int u0,
                                       int end, int g, int t) {
    using F = Frag<D, KV8>;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = u0 + 8 * (i >> 1) + 2 * t + (i & 1);
        const int key = u < end ? kl.row(u) : -1;
        const uint8_t* src = static_cast<const uint8_t*>(a.v) + (seq0 + key) * F::ROW;
        if (F::VB == 8) {
            const uint2 x = key >= 0 ? __ldg(reinterpret_cast<const uint2*>(src) + g) : make_uint2(0, 0);
            f.v[i][0] = x.x; f.v[i][1] = x.y;
        } else {
#pragma unroll
            for (int c = 0; c < F::VB / 16; ++c) {
                const uint4 x = key >= 0 ? __ldg(reinterpret_cast<const uint4*>(src) + g + 8 * c) : make_uint4(0, 0, 0, 0);
                f.v[i][4 * c % F::VW] = x.x; f.v[i][(4 * c + 1) % F::VW] = x.y;
                f.v[i][(4 * c + 2) % F::VW] = x.z; f.v[i][(4 * c + 3) % F::VW] = x.w;
            }
        }
        if (KV8) f.vs[i] = key >= 0 ? __ldg(a.v_scale + seq0 + key) : 0.f;
    }
}

// First of the 16 consecutive output dims of thread t that n-tiles 8c .. 8c+7 hold: dims
// +0..7 in the fragment's even column, +8..15 in the odd one (e4m3 rows of 128: 32 dims
// from 16 n-tiles, 16 per column).
template <int D, bool KV8>
__device__ __forceinline__ int out_dim(int nt, int col, int t) {
    return Frag<D, KV8>::VB == 16 && KV8 ? 16 * (2 * t + col) + nt : (nt >> 3) * 64 + 8 * (2 * t + col) + (nt & 7);
}

template <int D, bool KV8>
__global__ void __launch_bounds__(NW * 32, 1) window_rows_kernel(WindowArgs a) {
    using F = Frag<D, KV8>;
    constexpr int KS = D / 16;                   // k-steps of S
    constexpr int NT = D / 8;                    // n-tiles of O
    extern __shared__ float sm[];                // [NW][16][D] O, then [NW][16] max, [NW][16] sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tiles = (a.n_q * a.heads + 15) / 16;
    const int b = blockIdx.x / tiles, f0 = (blockIdx.x - b * tiles) * 16;
    const int split = blockIdx.y;
    const int live = live_rows(a.n_rows, b, a.n_q);
    if (f0 >= live * a.heads) return;
    const int base = checked_base(a.q_pos0, b, live, a.max_ctx, a.status);
    const int f_last = min(f0 + 15, live * a.heads - 1);
    const KeyList kl(base + f0 / a.heads, base + f_last / a.heads, a.window, a.sinks);
    const int chunk = ((kl.total + a.splits - 1) / a.splits + STEP - 1) / STEP * STEP;
    const int begin = min(kl.total, split * chunk), end = min(kl.total, begin + chunk);
    const int64_t seq0 = static_cast<int64_t>(b) * a.cap;
    const int64_t flat0 = static_cast<int64_t>(b) * a.n_q * a.heads;

    // Q fragments of pairs g and g + 8 in the keys' order of dims, and the pairs' positions
    uint32_t qa[KS][4];
    int pos[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int f = f0 + g + 8 * r;
        pos[r] = f <= f_last ? base + f / a.heads : -1;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (flat0 + f) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d = KV8 ? 16 * (t + 4 * (ks >> 2)) + 4 * (ks & 3) : 8 * (t + 4 * (ks >> 1)) + 4 * (ks & 1);
            const uint2 x = f <= f_last ? __ldg(reinterpret_cast<const uint2*>(q + d)) : make_uint2(0, 0);
            qa[ks][r] = x.x;
            qa[ks][2 + r] = x.y;
        }
    }

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const float sc2 = a.scale * kLog2e;

    F f;
    int u0 = begin + warp * STEP;
    if (u0 < end) {
        load_k(f, a, seq0, kl, u0, end, g, t);
        load_v(f, a, seq0, kl, u0, end, g, t);
    }
    for (; u0 < end; u0 += NW * STEP) {
        float s[2][4];
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
                        codes_to_bf16(w[i], b0, b1);
                        mma_bf16(s[h], qa[4 * c + i], b0, b1);
                    }
                } else {
                    mma_bf16(s[h], qa[2 * c], w[0], w[1]);
                    mma_bf16(s[h], qa[2 * c + 1], w[2], w[3]);
                }
            }
            // logits in log2 units, hidden keys at -inf
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = u0 + 8 * h + 2 * t + (j & 1);
                const int key = u < end ? kl.row(u) : -1;
                const float x = KV8 ? s[h][j] * f.ks[2 * h + (j & 1)] * sc2 : s[h][j] * sc2;
                s[h][j] = window_sees(key, pos[j >> 1], a.window, a.sinks) ? x : -INFINITY;
            }
        }
        const int un = u0 + NW * STEP;
        if (un < end) load_k(f, a, seq0, kl, un, end, g, t);
        float mn[2];
        bool rose = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float x = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            mn[r] = fmaxf(m[r], x);
            rose |= mn[r] > m[r];
        }
        if (__any_sync(0xffffffffu, rose)) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float c = mn[r] == -INFINITY ? 1.f : ex2(m[r] - mn[r]);
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
                float p0 = ex2(s[h][2 * r] - off), p1 = ex2(s[h][2 * r + 1] - off);
                l[r] += p0 + p1;
                if (KV8) {
                    p0 *= f.vs[2 * h];
                    p1 *= f.vs[2 * h + 1];
                }
                // P in bf16: one rounding of at most 2^-8 relative per weight, the MMA's operand type
                pa[2 * h + r] = pack_bf16(p0, p1);
            }
        if (KV8) {
            // bytes of keys (2t, 2t + 1) side by side, then widened
#pragma unroll
            for (int w = 0; w < F::VW; ++w)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t sel = q ? 0x7362u : 0x5140u;
                    uint32_t a0, a1, b0, b1;
                    codes_to_bf16(prmt(f.v[0][w], f.v[1][w], sel), a0, a1);
                    codes_to_bf16(prmt(f.v[2][w], f.v[3][w], sel), b0, b1);
                    mma_bf16(o[(4 * w + 2 * q) % NT], pa, a0, b0);
                    mma_bf16(o[(4 * w + 2 * q + 1) % NT], pa, a1, b1);
                }
        } else {
#pragma unroll
            for (int w = 0; w < F::VW; ++w) {
                mma_bf16(o[(2 * w) % NT], pa, prmt(f.v[0][w], f.v[1][w], 0x5410u), prmt(f.v[2][w], f.v[3][w], 0x5410u));
                mma_bf16(o[(2 * w + 1) % NT], pa, prmt(f.v[0][w], f.v[1][w], 0x7632u),
                         prmt(f.v[2][w], f.v[3][w], 0x7632u));
            }
        }
        if (un < end) load_v(f, a, seq0, kl, un, end, g, t);
    }

    // join the warps: pairs' maxima and sums, then O scaled to the common maximum
    float* so = sm;
    float* s_m = sm + NW * 16 * D;
    float* s_l = s_m + NW * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (t == 0) {
            s_m[warp * 16 + g + 8 * r] = m[r];
            s_l[warp * 16 + g + 8 * r] = l[r];
        }
    }
    const int active = min(NW, (end - begin + STEP - 1) / STEP);           // warps with keys
    if (warp < active) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                so[(warp * 16 + g + 8 * (j >> 1)) * D + out_dim<D, KV8>(i, j & 1, t)] = o[i][j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * D / 4; i += NW * 32) {
        const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
        if (f0 + r > f_last) continue;
        float mx = -INFINITY;
        for (int w = 0; w < active; ++w) mx = fmaxf(mx, s_m[w * 16 + r]);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < active; ++w) {
            const float mw = s_m[w * 16 + r];
            const float c = mw == -INFINITY ? 0.f : ex2(mw - mx);
            const float4 x = *reinterpret_cast<const float4*>(so + (w * 16 + r) * D + d);
            sum = fmaf(c, s_l[w * 16 + r], sum);
            acc.x = fmaf(c, x.x, acc.x); acc.y = fmaf(c, x.y, acc.y);
            acc.z = fmaf(c, x.z, acc.z); acc.w = fmaf(c, x.w, acc.w);
        }
        const int64_t flat = flat0 + f0 + r;
        if (a.splits == 1) {
            const float inv = 1.f / sum;
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + flat * D + d) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
            if (a.lse && d == 0) a.lse[flat] = (mx + log2f(sum)) * kLn2;
        } else {
            const int64_t at = static_cast<int64_t>(split) * a.batch * a.n_q * a.heads + flat;
            *reinterpret_cast<float4*>(a.part_o + at * D + d) = acc;
            if (d == 0) a.part_ml[at] = make_float2(mx, sum);
        }
    }
}

// fp32: 64 pairs x 32 keys per tile on the CUDA cores (a bf16 or tf32 product would lose
// what the fp32 caches are there for).  Thread (rp, qt) of 32 x 4 has pairs 2 rp, 2 rp + 1;
// keys qt + 4 i of S, dims 4 qt + 16 i of O: nine or ten 16-byte shared loads per 64 FMAs.
template <int D>
__global__ void __launch_bounds__(128) window_f32_kernel(WindowArgs a) {
    constexpr int LDQ = D + 4;                   // row pitch: rows of a quarter-warp on distinct banks
    constexpr int NC = D / 16;                   // float4 chunks of O per thread and pair
    extern __shared__ float4 sm4[];
    float* sq = reinterpret_cast<float*>(sm4);   // [64][LDQ]
    float* sk = sq + F_ROWS * LDQ;               // [32][LDQ]
    float* sv = sk + F_KEYS * LDQ;               // [32][D]
    float* sp = sv + F_KEYS * D;                 // [64][33]
    const int tid = threadIdx.x, rp = tid >> 2, qt = tid & 3;
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

    for (int i = tid; i < F_ROWS * D / 4; i += 128) {
        const int r = i / (D / 4), c = i - r * (D / 4);
        const float4 x = f0 + r <= f_last ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (flat0 + f0 + r) * D) + c)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(sq + r * LDQ + 4 * c) = x;
    }
    int pos[2];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float4 o[2][NC];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int f = f0 + 2 * rp + r;
        pos[r] = f <= f_last ? base + f / a.heads : -1;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int u0 = begin; u0 < end; u0 += F_KEYS) {
        __syncthreads();
        for (int i = tid; i < F_KEYS * D / 4; i += 128) {
            const int r = i / (D / 4), c = i - r * (D / 4);
            const int key = u0 + r < end ? kl.row(u0 + r) : -1;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            if (key >= 0) {
                x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.k) + (seq0 + key) * D) + c);
                y = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.v) + (seq0 + key) * D) + c);
            }
            *reinterpret_cast<float4*>(sk + r * LDQ + 4 * c) = x;
            *reinterpret_cast<float4*>(sv + r * D + 4 * c) = y;
        }
        __syncthreads();
        float s[2][8];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[r][i] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 4; ++c) {
            const float4 x0 = *reinterpret_cast<const float4*>(sq + (2 * rp) * LDQ + 4 * c);
            const float4 x1 = *reinterpret_cast<const float4*>(sq + (2 * rp + 1) * LDQ + 4 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(sk + (qt + 4 * i) * LDQ + 4 * c);
                s[0][i] = fmaf(x0.x, y.x, fmaf(x0.y, y.y, fmaf(x0.z, y.z, fmaf(x0.w, y.w, s[0][i]))));
                s[1][i] = fmaf(x1.x, y.x, fmaf(x1.y, y.y, fmaf(x1.z, y.z, fmaf(x1.w, y.w, s[1][i]))));
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int u = u0 + qt + 4 * i;
                const int key = u < end ? kl.row(u) : -1;
                s[r][i] = window_sees(key, pos[r], a.window, a.sinks) ? s[r][i] * sc2 : -INFINITY;
                mx = fmaxf(mx, s[r][i]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[r], mx);
            const float c = mn == -INFINITY ? 1.f : exp2f(m[r] - mn), off = mn == -INFINITY ? 0.f : mn;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = exp2f(s[r][i] - off);
                sum += p;
                sp[(2 * rp + r) * 33 + qt + 4 * i] = p;
            }
            l[r] = fmaf(l[r], c, sum);
            m[r] = mn;
#pragma unroll
            for (int j = 0; j < NC; ++j) { o[r][j].x *= c; o[r][j].y *= c; o[r][j].z *= c; o[r][j].w *= c; }
        }
        __syncwarp();                            // a pair's weights come from the four threads of its quad
#pragma unroll 4
        for (int k = 0; k < F_KEYS; ++k) {
            const float p0 = sp[(2 * rp) * 33 + k], p1 = sp[(2 * rp + 1) * 33 + k];
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(sv + k * D + 4 * qt + 16 * j);
                o[0][j].x = fmaf(p0, y.x, o[0][j].x); o[0][j].y = fmaf(p0, y.y, o[0][j].y);
                o[0][j].z = fmaf(p0, y.z, o[0][j].z); o[0][j].w = fmaf(p0, y.w, o[0][j].w);
                o[1][j].x = fmaf(p1, y.x, o[1][j].x); o[1][j].y = fmaf(p1, y.y, o[1][j].y);
                o[1][j].z = fmaf(p1, y.z, o[1][j].z); o[1][j].w = fmaf(p1, y.w, o[1][j].w);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const int f = f0 + 2 * rp + r;
        if (f > f_last) continue;
        const int64_t flat = flat0 + f;
        const int64_t at = static_cast<int64_t>(blockIdx.y) * a.batch * a.n_q * a.heads + flat;
        const float inv = a.splits == 1 ? 1.f / l[r] : 1.f;
        float* dst = a.splits == 1 ? static_cast<float*>(a.o) + flat * D : a.part_o + at * D;
#pragma unroll
        for (int j = 0; j < NC; ++j)
            *reinterpret_cast<float4*>(dst + 4 * qt + 16 * j) =
                make_float4(o[r][j].x * inv, o[r][j].y * inv, o[r][j].z * inv, o[r][j].w * inv);
        if (qt == 0) {
            if (a.splits > 1) a.part_ml[at] = make_float2(m[r], l[r]);
            else if (a.lse) a.lse[flat] = (m[r] + log2f(l[r])) * kLn2;
        }
    }
}

// Joins the parts of a pair: one warp per pair, D / 32 dims per lane, parts in order.
template <typename T, int D>
__global__ void __launch_bounds__(128) window_join_kernel(WindowArgs a) {
    constexpr int PER = D / 32;
    const int64_t all = static_cast<int64_t>(a.batch) * a.n_q * a.heads;
    const int64_t flat = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (flat >= all) return;
    const int64_t row = flat / a.heads;
    const int b = static_cast<int>(row / a.n_q);
    if (row - static_cast<int64_t>(b) * a.n_q >= live_rows(a.n_rows, b, a.n_q)) return;
    float mx = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) mx = fmaxf(mx, a.part_ml[s * all + flat].x);
    mx = warp_max(mx);
    float sum = 0.f, acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const float2 ml = a.part_ml[s * all + flat];
        float x[PER];
        const float* src = a.part_o + (s * all + flat) * D + lane * PER;
        if (PER == 4) {
            const float4 y = *reinterpret_cast<const float4*>(src);
            x[0] = y.x; x[1] = y.y; x[2 % PER] = y.z; x[3 % PER] = y.w;
        } else {
            const float2 y = *reinterpret_cast<const float2*>(src);
            x[0] = y.x; x[1] = y.y;
        }
        const bool some = ml.x != -INFINITY;         // a part without keys may have left no O
        const float c = some ? exp2f(ml.x - mx) : 0.f;
        sum = fmaf(c, ml.y, sum);
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = fmaf(c, some ? x[i] : 0.f, acc[i]);
    }
    const float inv = 1.f / sum;
    T* dst = static_cast<T*>(a.o) + flat * D + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) dst[i] = static_cast<T>(acc[i] * inv);
    if (a.lse && lane == 0) a.lse[flat] = (mx + log2f(sum)) * kLn2;
}

template <int D, bool KV8>
cudaError_t launch_rows(const WindowArgs& a, cudaStream_t st) {
    constexpr int smem = (NW * 16 * D + 2 * NW * 16) * 4;
    const cudaError_t e = cudaFuncSetAttribute(window_rows_kernel<D, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (static_cast<unsigned>(a.n_q) * a.heads + 15) / 16;
    window_rows_kernel<D, KV8><<<dim3(tiles * a.batch, a.splits), NW * 32, smem, st>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_f32(const WindowArgs& a, cudaStream_t st) {
    constexpr int smem = ((F_ROWS + F_KEYS) * (D + 4) + F_KEYS * D + F_ROWS * 33) * 4;
    const cudaError_t e = cudaFuncSetAttribute(window_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (static_cast<unsigned>(a.n_q) * a.heads + F_ROWS - 1) / F_ROWS;
    window_f32_kernel<D><<<dim3(tiles * a.batch, a.splits), 128, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_join(const WindowArgs& a, cudaStream_t st) {
    const int64_t all = static_cast<int64_t>(a.batch) * a.n_q * a.heads;
    window_join_kernel<T, D><<<static_cast<unsigned>((all + 3) / 4), 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

WindowPlan plan_window(int batch, int n_q, int heads, int kv_dtype, int window, int sinks, int64_t max_ctx) {
    const bool f32 = kv_dtype == HS2_F32;
    const int64_t pairs = static_cast<int64_t>(n_q) * heads;
    WindowPlan p{};
    p.tile = !f32 && pairs >= kTilePairs;
    const int rows = f32 ? F_ROWS : (p.tile ? 256 : 16);
    const int64_t tiles = (pairs + rows - 1) / rows * batch;
    // keys of a tile: its rows' windows and the sinks, at most the whole context
    int64_t keys = static_cast<int64_t>(window) + rows / heads + sinks + kSinkPad;
    if (keys > max_ctx + kSinkPad) keys = max_ctx + kSinkPad;
    // parts: as many as fill the SMs once, each with enough keys to be worth the join
    int64_t s = num_sms() * (f32 ? 2 : 1) / tiles;
    const int64_t most = keys / (f32 ? kMinSplitKeysF32 : kMinSplitKeys);
    if (s > most) s = most;
    p.splits = s < 1 ? 1 : static_cast<int>(s);
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
