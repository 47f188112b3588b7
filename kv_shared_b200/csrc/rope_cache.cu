// rope_cache.cu -- norm of each query head and of the key, position rotation, and the
// write of the key and value rows to the cache, in one pass over the rows.
//
// Per head x of a row:  y = x rsqrt(mean(x^2) + eps) w;  each pair (a, b) of the first
// rot_dim dims turns by pos * inv_freq:  (a cos - b sin, b cos + a sin).
//
// Bound by HBM: a row reads (H + 2) D values and writes H D plus two cache rows, a few
// operations per value; what has to stay small is everything per vector that is not the
// vector.  A warp takes a row (with few rows, a part of its heads), D / 8 lanes to a vector
// with 8 dims (16 B of bf16) to a lane, UN vectors in flight per lane.  A lane's weights and
// angles are multiplied once and serve every query head of the row, two dims to an
// instruction; the key and the value, one of each, go their own way at the end.  (All vectors
// on one path, chosen by selection: 86 us for 4 x 8192 rows of 16 heads of 128.)  The angles
// depend on the row alone and are formed by its warp: position times frequency in turns in fp64, the
// whole turns dropped there, so that a position of a million loses nothing, then sine and cosine of
// the fraction in fp32.  Measured, replayed from a graph on the same inputs: 4 x 8192 rows of 16 heads
// of 128 56.8 us (5.3 TB/s), 32 single rows 3.2 us; as calls among others on changing inputs 61.4 and 4.5.
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"

namespace hs2 {
namespace {

constexpr int NT = 128;
constexpr int NW = NT / 32;
constexpr int UN = 2;                            // query vectors in flight per lane

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

// The 8 dims of a lane: two groups of four, at d0 and d1.  Plain loads: q_out may be q, and the
// read-only path is for memory that the kernel does not write.
__device__ __forceinline__ void load8(Raw<__nv_bfloat16>& r, const __nv_bfloat16* x, int d0, int d1, bool together) {
    if (together) {
        r.a = *reinterpret_cast<const uint4*>(x + d0);
    } else {
        const uint2 p = *reinterpret_cast<const uint2*>(x + d0), q = *reinterpret_cast<const uint2*>(x + d1);
        r.a = make_uint4(p.x, p.y, q.x, q.y);
    }
}
__device__ __forceinline__ void load8(Raw<float>& r, const float* x, int d0, int d1, bool) {
    r.a = *reinterpret_cast<const float4*>(x + d0);
    r.b = *reinterpret_cast<const float4*>(x + d1);
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
// wpr: warps that share a row (1 or NW); blocks: CTAs per sequence.
template <typename T, typename TC, bool E4, int D, int MODE>
__global__ void __launch_bounds__(NT) rope_cache_kernel(RopeArgs a, int wpr, int blocks) {
    constexpr int LPV = D / 8;                   // lanes per vector
    constexpr int VPW = 32 / LPV;                // vectors per warp
    constexpr bool TOGETHER = MODE != HALVES;
    __shared__ float2 tab[NW][D / 2];            // (cos, sin) of each warp's row
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / blocks;
    const int r = wpr == 1 ? (blockIdx.x - b * blocks) * NW + warp : blockIdx.x - b * blocks;
    if (r >= (a.n_rows ? min(a.n_rows[b], a.n) : a.n)) return;
    const int64_t row = static_cast<int64_t>(b) * a.n + r;
    const int64_t at = static_cast<int64_t>(a.row0[b]) + r;     // cache row
    const int rot = MODE == HALVES ? D : a.rot, half = rot >> 1;
    const int l = lane % LPV;                    // lane within the vector
    const int d0 = TOGETHER ? 8 * l : 4 * l;
    const int d1 = TOGETHER ? d0 + 4 : d0 + D / 2;
    // the first vectors are on their way while the angles are formed, the next ones while one is turned
    const int heads = a.q ? a.heads : 0, step = (wpr == 1 ? 1 : NW) * VPW, u00 = wpr == 1 ? 0 : warp * VPW;
    const T* q = static_cast<const T*>(a.q) + row * a.q_row;
    Raw<T> raw[UN], kv{};
    auto load_q = [&](int u0) {
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int head = u0 + u * step + lane / LPV;
            if (head < heads) load8(raw[u], q + head * D, d0, d1, TOGETHER);
        }
    };
#pragma unroll
    for (int u = 0; u < UN; ++u) raw[u] = Raw<T>{};
    load_q(u00);
    // the key in the first lanes of a warp, the value in the next
    const bool kv_warp = wpr == 1 || warp == NW - 1;
    const bool is_k = lane / LPV == 0 && a.k && kv_warp, is_v = lane / LPV == 1 && a.v && kv_warp;
    if (is_k) load8(kv, static_cast<const T*>(a.k) + row * a.k_row, d0, d1, TOGETHER);
    if (is_v) load8(kv, static_cast<const T*>(a.v) + row * a.v_row, d0, d1, TOGETHER);
    {
        const double p = a.pos ? a.pos[row] : static_cast<double>(at);
        for (int j = lane; j < half; j += 32) {
            const double turns = p * (a.inv_freq[j] * 0.15915494309189533577);  // 1 / (2 pi)
            float s, c;
            sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
            tab[warp][j] = make_float2(c, s);
        }
        __syncwarp();
    }
    // dims past rot (a multiple of 16: all eight of a lane) keep their partners out, 0 * infinity being NaN
    const bool still = MODE != HALVES && d0 >= rot;
    // PARTIAL: the partner's lane, half a rotation (a multiple of 8 dims) up or down
    const int from = MODE == PARTIAL && d0 < rot ? lane + (d0 < half ? half >> 3 : -(half >> 3)) : lane;
    // out[i] = inv (x[i] c[i] + x[partner of i] s[i]): cosine and signed sine times the weights
    float2 c[4], s[4];
    auto coefficients = [&](const float* w) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = i < 4 ? d0 + i : d1 + i - 4;
            const bool turns = d < rot, high = MODE == ADJACENT ? d & 1 : d >= half;
            const int pair = MODE == ADJACENT ? d >> 1 : (high ? d - half : d);
            const int other = MODE == ADJACENT ? d ^ 1 : (high ? d - half : d + half);
            const float2 t = turns ? tab[warp][pair] : make_float2(1.f, 0.f);
            const float wd = w ? __ldg(w + d) : 1.f, wo = w && turns ? __ldg(w + other) : 1.f;
            (i & 1 ? c[i / 2].y : c[i / 2].x) = t.x * wd;
            (i & 1 ? s[i / 2].y : s[i / 2].x) = (high ? t.y : -t.y) * wo;
        }
    };
    // a vector's eight dims in a lane: normed and turned
    auto turn = [&](const Raw<T>& raw, float (&x)[8]) {
        float y[8], o[8];
        widen(raw, y);
        if (MODE == PARTIAL) {
            Raw<T> far;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(&raw);
            uint32_t* dst = reinterpret_cast<uint32_t*>(&far);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(Raw<T>) / 4); ++i) dst[i] = __shfl_sync(0xffffffffu, src[i], from);
            widen(far, o);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = MODE == ADJACENT ? y[i ^ 1] : y[i ^ 4];
        }
        float inv = 1.f;
        if (a.normalize) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; i += 2) ss = fma2(make_float2(y[i], y[i + 1]), make_float2(y[i], y[i + 1]), ss);
            float sum = ss.x + ss.y;
#pragma unroll
            for (int k = LPV / 2; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            inv = rsqrtf(sum * (1.f / D) + a.eps);
        }
        const float2 z = make_float2(0.f, 0.f), i2 = make_float2(inv, inv);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float2 t = fma2(make_float2(y[i], y[i + 1]), c[i / 2], z);
            if (!still) t = fma2(make_float2(o[i], o[i + 1]), s[i / 2], t);
            t = fma2(t, i2, z);
            x[i] = t.x;
            x[i + 1] = t.y;
        }
    };

    if (heads > 0) {
        coefficients(a.normalize ? a.q_weight : nullptr);
        T* qo = static_cast<T*>(a.q_out) + row * a.heads * D;
        for (int u0 = u00; u0 < heads; u0 += UN * step) {
            Raw<T> now[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u) now[u] = raw[u];
            load_q(u0 + UN * step);
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int head = u0 + u * step + lane / LPV;
                if (u0 + u * step < heads) {                    // the whole warp
                    float x[8];
                    turn(now[u], x);
                    if (head < heads) store8(qo + head * D, d0, d1, TOGETHER, x);
                }
            }
        }
    }
    if (!kv_warp || (!a.k && !a.v)) return;
    coefficients(a.normalize ? a.k_weight : nullptr);
    float x[8], y[8];
    turn(kv, x);
    widen(kv, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = is_v ? y[i] : x[i];
    float amax = 0.f;
    if (E4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int o = LPV / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if ((!is_k && !is_v) || at < 0 || at >= a.cap) return;
    const int64_t dst = b * a.cap + at;
    if (E4) {
        const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], sc);
        uint8_t* p = static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) + dst * D;
        const uint32_t lo = e4m3x4(x[0], x[1], x[2], x[3]), hi = e4m3x4(x[4], x[5], x[6], x[7]);
        if (TOGETHER) {
            *reinterpret_cast<uint2*>(p + d0) = make_uint2(lo, hi);
        } else {
            *reinterpret_cast<uint32_t*>(p + d0) = lo;
            *reinterpret_cast<uint32_t*>(p + d1) = hi;
        }
        if (l == 0) (is_k ? a.k_scale : a.v_scale)[dst] = sc;
    } else {
        store8(static_cast<TC*>(is_k ? a.k_cache : a.v_cache) + dst * D, d0, d1, TOGETHER, x);
    }
}

template <typename T, typename TC, bool E4, int D>
cudaError_t launch_mode(const RopeArgs& a, int wpr, int blocks, cudaStream_t st) {
    const dim3 g(static_cast<unsigned>(blocks) * a.batch);
    if (a.interleaved || a.rot == 0) rope_cache_kernel<T, TC, E4, D, ADJACENT><<<g, NT, 0, st>>>(a, wpr, blocks);
    else if (a.rot == D) rope_cache_kernel<T, TC, E4, D, HALVES><<<g, NT, 0, st>>>(a, wpr, blocks);
    else rope_cache_kernel<T, TC, E4, D, PARTIAL><<<g, NT, 0, st>>>(a, wpr, blocks);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_type(const RopeArgs& a, int wpr, int blocks, cudaStream_t st) {
    if (a.in_f32) {
        if (a.kv_dtype == HS2_F32) return launch_mode<float, float, false, D>(a, wpr, blocks, st);
        if (a.kv_dtype == HS2_BF16) return launch_mode<float, __nv_bfloat16, false, D>(a, wpr, blocks, st);
        return launch_mode<float, float, true, D>(a, wpr, blocks, st);
    }
    if (a.kv_dtype == HS2_BF16) return launch_mode<__nv_bfloat16, __nv_bfloat16, false, D>(a, wpr, blocks, st);
    return launch_mode<__nv_bfloat16, __nv_bfloat16, true, D>(a, wpr, blocks, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.batch) * a.n;
    // a warp per row once that gives every SM a CTA; before, a CTA per row (the call is then as
    // short as its slowest warp)
    const int wpr = rows >= static_cast<int64_t>(NW) * num_sms() ? 1 : NW;
    const int blocks = wpr == 1 ? (a.n + NW - 1) / NW : a.n;
    return a.head_dim == 128 ? launch_type<128>(a, wpr, blocks, st) : launch_type<64>(a, wpr, blocks, st);
}

}  // namespace hs2
