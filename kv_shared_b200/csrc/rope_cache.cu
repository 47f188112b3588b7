// rope_cache.cu -- norm of each query head and of the key, position rotation, and the
// write of the key and value rows to the cache, in one pass over the rows.
//
// Per head x of a row:  y = x rsqrt(mean(x^2) + eps) w;  each pair (a, b) of the first
// rot_dim dims turns by pos * inv_freq:  (a cos - b sin, b cos + a sin).
//
// Bound by HBM: a row reads (H + 2) D values and writes H D plus two cache rows, a few
// operations per value.  A CTA takes TOK rows; its (row, head) vectors are spread over the
// warps, D / 8 lanes to a vector with 8 dims (16 B of bf16) to a lane, four vectors in
// flight per lane so that the loads cover the memory latency.  The angles depend on the
// row alone and are formed once per CTA into shared memory (computed by every vector they
// would cost as much as the rest): position times frequency in turns in fp64, the whole
// turns dropped there, so that a position of a million loses nothing, then sine and
// cosine of the fraction in fp32.
#include "common.cuh"
#include "internal.h"

namespace hs2 {
namespace {

constexpr int NT = 256;
constexpr int UN = 4;                            // vectors in flight per lane

enum { ADJACENT = 0, HALVES = 1, PARTIAL = 2 };  // pairs (2i, 2i+1); (i, i+D/2); (i, i+rot/2), rot < D

template <typename T>
struct Raw {};
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Raw<float> {
    float4 a, b;
};

// The 8 dims of a lane: two groups of four, at d0 and d1.
__device__ __forceinline__ void load8(Raw<__nv_bfloat16>& r, const __nv_bfloat16* x, int d0, int d1, bool together) {
    if (together) {
        r.a = __ldg(reinterpret_cast<const uint4*>(x + d0));
    } else {
        const uint2 p = __ldg(reinterpret_cast<const uint2*>(x + d0)), q = __ldg(reinterpret_cast<const uint2*>(x + d1));
        r.a = make_uint4(p.x, p.y, q.x, q.y);
    }
}
__device__ __forceinline__ void load8(Raw<float>& r, const float* x, int d0, int d1, bool) {
    r.a = __ldg(reinterpret_cast<const float4*>(x + d0));
    r.b = __ldg(reinterpret_cast<const float4*>(x + d1));
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&v)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&v)[8]) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* x, int d0, int d1, bool together, const float (&v)[8]) {
    const uint2 p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    const uint2 q = make_uint2(pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    if (together) {
        *reinterpret_cast<uint4*>(x + d0) = make_uint4(p.x, p.y, q.x, q.y);
    } else {
        *reinterpret_cast<uint2*>(x + d0) = p;
        *reinterpret_cast<uint2*>(x + d1) = q;
    }
}
__device__ __forceinline__ void store8(float* x, int d0, int d1, bool, const float (&v)[8]) {
    *reinterpret_cast<float4*>(x + d0) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(x + d1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    // the second source operand lands in the low byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// T: type of q, k, v and q_out; TC: type of the cache rows, unless E4 (e4m3 codes and scales).
template <typename T, typename TC, bool E4, int D, int MODE>
__global__ void __launch_bounds__(NT) rope_cache_kernel(RopeArgs a, int tok) {
    constexpr int LPV = D / 8;                   // lanes per vector
    constexpr int VPW = 32 / LPV;                // vectors per warp
    constexpr bool TOGETHER = MODE != HALVES;
    extern __shared__ float2 tab[];              // [tok][rot / 2] (cos, sin)
    const int half = a.rot >> 1;
    const int64_t rows = static_cast<int64_t>(a.batch) * a.n;
    const int64_t row_base = static_cast<int64_t>(blockIdx.x) * tok;
    const int here = static_cast<int>(rows - row_base < tok ? rows - row_base : tok);

    for (int i = threadIdx.x; i < here * half; i += NT) {
        const int t = i / half, j = i - t * half;
        const int64_t row = row_base + t;
        const int b = static_cast<int>(row / a.n);
        const int p = a.pos ? a.pos[row] : a.row0[b] + static_cast<int>(row - static_cast<int64_t>(b) * a.n);
        const double turns = p * (a.inv_freq[j] * 0.15915494309189533577);      // 1 / (2 pi)
        float s, c;
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
        tab[i] = make_float2(c, s);
    }
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPV;                    // lane within the vector
    const int d0 = TOGETHER ? 8 * l : 4 * l;
    const int d1 = TOGETHER ? d0 + 4 : d0 + D / 2;
    const int nq = a.q ? a.heads : 0, nk = a.k ? 1 : 0;
    const int nvec = nq + nk + (a.v ? 1 : 0);
    const int total = here * nvec;
    for (int u0 = warp * VPW * UN; u0 < total; u0 += (NT / 32) * VPW * UN) {
        Raw<T> raw[UN];
        int tt[UN], kind[UN];                    // row of the CTA; head, or nq (key), nq + 1 (value); -1: none
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int unit = u0 + u * VPW + lane / LPV;
            kind[u] = -1;
            tt[u] = 0;
            raw[u] = Raw<T>{};
            if (unit < total) {
                const int t = unit / nvec, vec = unit - t * nvec;
                const int64_t row = row_base + t;
                const int b = static_cast<int>(row / a.n);
                const int r = static_cast<int>(row - static_cast<int64_t>(b) * a.n);
                if (!a.n_rows || r < a.n_rows[b]) {
                    kind[u] = vec < nq ? vec : (vec == nq && nk ? nq : nq + 1);
                    tt[u] = t;
                    const T* src = vec < nq ? static_cast<const T*>(a.q) + row * a.q_row + vec * D
                                            : (kind[u] == nq ? static_cast<const T*>(a.k) + row * a.k_row
                                                             : static_cast<const T*>(a.v) + row * a.v_row);
                    load8(raw[u], src, d0, d1, TOGETHER);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const bool is_v = kind[u] == nq + 1, is_k = kind[u] == nq;
            float v[8];
            widen(raw[u], v);
            // every lane takes the shuffles; what does not apply to values is undone by selection
            if (a.normalize) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
                for (int o = LPV / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = is_v ? 1.f : rsqrtf(ss * (1.f / D) + a.eps);
                const float* w = is_k ? a.k_weight : a.q_weight;
                if (w && !is_v) {
                    const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + d0));
                    const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + d1));
                    v[0] *= inv * w0.x; v[1] *= inv * w0.y; v[2] *= inv * w0.z; v[3] *= inv * w0.w;
                    v[4] *= inv * w1.x; v[5] *= inv * w1.y; v[6] *= inv * w1.z; v[7] *= inv * w1.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= inv;
                }
            }
            const float2* cs = tab + tt[u] * half;
            if (MODE == ADJACENT) {
                if (d0 < a.rot && !is_v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = cs[(d0 >> 1) + i];
                        const float x = v[2 * i], y = v[2 * i + 1];
                        v[2 * i] = x * t.x - y * t.y;
                        v[2 * i + 1] = y * t.x + x * t.y;
                    }
                }
            } else if (MODE == HALVES) {
                if (!is_v) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = cs[d0 + i];
                        const float x = v[i], y = v[4 + i];
                        v[i] = x * t.x - y * t.y;
                        v[4 + i] = y * t.x + x * t.y;
                    }
                }
            } else {
                // partner lane: half a rotation (a multiple of 8 dims) up or down
                const bool low = d0 < half;
                const int step = half >> 3;
                const int from = d0 < a.rot ? lane + (low ? step : -step) : lane;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, v[i], from);
                if (d0 < a.rot && !is_v) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 t = cs[(low ? d0 : d0 - half) + i];
                        v[i] = low ? v[i] * t.x - o[i] * t.y : v[i] * t.x + o[i] * t.y;
                    }
                }
            }
            float amax = 0.f;
            if (E4) {
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
                for (int o = LPV / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            }
            if (kind[u] < 0) continue;
            const int64_t row = row_base + tt[u];
            if (kind[u] < nq) {
                store8(static_cast<T*>(a.q_out) + (row * a.heads + kind[u]) * D, d0, d1, TOGETHER, v);
                continue;
            }
            const int b = static_cast<int>(row / a.n);
            const int64_t at = static_cast<int64_t>(a.row0[b]) + (row - static_cast<int64_t>(b) * a.n);
            if (at < 0 || at >= a.cap) continue;
            const int64_t dst = b * a.cap + at;
            if (E4) {
                const float s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], s);
                uint8_t* c = static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) + dst * D;
                const uint32_t lo = e4m3x4(v[0], v[1], v[2], v[3]), hi = e4m3x4(v[4], v[5], v[6], v[7]);
                if (TOGETHER) {
                    *reinterpret_cast<uint2*>(c + d0) = make_uint2(lo, hi);
                } else {
                    *reinterpret_cast<uint32_t*>(c + d0) = lo;
                    *reinterpret_cast<uint32_t*>(c + d1) = hi;
                }
                if (l == 0) (is_k ? a.k_scale : a.v_scale)[dst] = s;
            } else {
                store8(static_cast<TC*>(is_k ? a.k_cache : a.v_cache) + dst * D, d0, d1, TOGETHER, v);
            }
        }
    }
}

template <typename T, typename TC, bool E4, int D>
cudaError_t launch_mode(const RopeArgs& a, int tok, int64_t grid, cudaStream_t st) {
    const size_t smem = sizeof(float2) * tok * (a.rot >> 1);
    const dim3 g(static_cast<unsigned>(grid));
    if (a.interleaved || a.rot == 0) rope_cache_kernel<T, TC, E4, D, ADJACENT><<<g, NT, smem, st>>>(a, tok);
    else if (a.rot == D) rope_cache_kernel<T, TC, E4, D, HALVES><<<g, NT, smem, st>>>(a, tok);
    else rope_cache_kernel<T, TC, E4, D, PARTIAL><<<g, NT, smem, st>>>(a, tok);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_type(const RopeArgs& a, int tok, int64_t grid, cudaStream_t st) {
    if (a.in_f32) {
        if (a.kv_dtype == HS2_F32) return launch_mode<float, float, false, D>(a, tok, grid, st);
        if (a.kv_dtype == HS2_BF16) return launch_mode<float, __nv_bfloat16, false, D>(a, tok, grid, st);
        return launch_mode<float, float, true, D>(a, tok, grid, st);
    }
    if (a.kv_dtype == HS2_BF16) return launch_mode<__nv_bfloat16, __nv_bfloat16, false, D>(a, tok, grid, st);
    return launch_mode<__nv_bfloat16, __nv_bfloat16, true, D>(a, tok, grid, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.batch) * a.n;
    // rows per CTA: one while that fills fewer than four CTAs per SM (the call is then as
    // short as its slowest CTA), up to eight (which share the angles' cost per thread)
    int tok = 1;
    while (tok < 8 && rows / (2 * tok) >= 4 * num_sms()) tok *= 2;
    const int64_t grid = (rows + tok - 1) / tok;
    return a.head_dim == 128 ? launch_type<128>(a, tok, grid, st) : launch_type<64>(a, tok, grid, st);
}

}  // namespace hs2
