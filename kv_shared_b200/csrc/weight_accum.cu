// weight_accum.cu -- accumulated attention weight of the cached keys.
//
//   acc_out[j] = decay acc_in[j] + sum over rows r and heads h of
//                exp(scale q_rh . k_j - lse_rh)            [j <= p_r]
//
// The log-sum-exp is known, so one product S = K Q^T and one exponential per (key, row,
// head) are all there is; the keys stay put and the (row, head) pairs stream past, so that
// a key's total is a sum inside a thread and no key is read twice.
#include "common.cuh"
#include "internal.h"
#include "window_keys.cuh"

namespace hs2 {
namespace {

constexpr int S_KEYS = 64;                       // keys per CTA
constexpr int S_ROWS = 32;                       // (row, head) pairs per tile

// Rows of a cache or of Q as four numbers.
__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const uint8_t* p) {
    const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(p));
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(x, lo, hi);
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&lo)), h = __half22float2(*reinterpret_cast<__half2*>(&hi));
    return make_float4(f.x, f.y, h.x, h.y);
}

// CUDA cores, fp32 arithmetic.  Thread (kp, qt) of 32 x 4 has keys 2 kp, 2 kp + 1 and the
// pairs qt + 4 i of a tile.
template <typename TQ, typename TK, int D>
__global__ void __launch_bounds__(128) accum_simt_kernel(AccumArgs a) {
    constexpr int LD = D + 4;
    extern __shared__ float4 sm4[];
    float* sk = reinterpret_cast<float*>(sm4);   // [64][LD]
    float* sq = sk + S_KEYS * LD;                // [32][LD]
    __shared__ float s_lse[S_ROWS];
    __shared__ int s_pos[S_ROWS];
    const int tid = threadIdx.x, kp = tid >> 2, qt = tid & 3;
    const int tiles = static_cast<int>((a.max_ctx + S_KEYS - 1) / S_KEYS);
    const int b = blockIdx.x / tiles, j0 = (blockIdx.x - b * tiles) * S_KEYS;
    const int live = live_rows(a.n_rows, b, a.n_q);
    const int base = checked_base(a.q_pos0, b, live, a.max_ctx, a.status);
    if (j0 >= base + live) return;
    const int64_t seq0 = static_cast<int64_t>(b) * a.cap;
    const int64_t flat0 = static_cast<int64_t>(b) * a.n_q * a.heads;
    const int flats = live * a.heads;
    const int chunk = ((flats + a.splits - 1) / a.splits + S_ROWS - 1) / S_ROWS * S_ROWS;
    // rows at positions before the tile's first key see none of its keys
    const int first = max(static_cast<int>(blockIdx.y) * chunk, max(0, j0 - base) * a.heads / S_ROWS * S_ROWS);
    const int end = min(flats, (static_cast<int>(blockIdx.y) + 1) * chunk);
    const float sc2 = a.scale * kLog2e;

    for (int i = tid; i < S_KEYS * D / 4; i += 128) {
        const int r = i / (D / 4), c = i - r * (D / 4);
        const float4 x = j0 + r < base + live ? load4(static_cast<const TK*>(a.k) + (seq0 + j0 + r) * D + 4 * c)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(sk + r * LD + 4 * c) = x;
    }
    float ksc[2], total[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int j = j0 + 2 * kp + r;
        ksc[r] = a.k_scale && j < base + live ? sc2 * a.k_scale[seq0 + j] : sc2;
    }
    for (int f0 = first; f0 < end; f0 += S_ROWS) {
        __syncthreads();
        for (int i = tid; i < S_ROWS * D / 4; i += 128) {
            const int r = i / (D / 4), c = i - r * (D / 4);
            const float4 x = f0 + r < end ? load4(static_cast<const TQ*>(a.q) + (flat0 + f0 + r) * D + 4 * c)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(sq + r * LD + 4 * c) = x;
        }
        if (tid < S_ROWS) {
            const int f = f0 + tid;
            s_lse[tid] = f < end ? a.lse[flat0 + f] * kLog2e : 0.f;
            s_pos[tid] = f < end ? base + f / a.heads : -1;
        }
        __syncthreads();
        float s[2][8];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[r][i] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 4; ++c) {
            const float4 x0 = *reinterpret_cast<const float4*>(sk + (2 * kp) * LD + 4 * c);
            const float4 x1 = *reinterpret_cast<const float4*>(sk + (2 * kp + 1) * LD + 4 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(sq + (qt + 4 * i) * LD + 4 * c);
                s[0][i] = fmaf(x0.x, y.x, fmaf(x0.y, y.y, fmaf(x0.z, y.z, fmaf(x0.w, y.w, s[0][i]))));
                s[1][i] = fmaf(x1.x, y.x, fmaf(x1.y, y.y, fmaf(x1.z, y.z, fmaf(x1.w, y.w, s[1][i]))));
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int p = s_pos[qt + 4 * i];
            const float off = s_lse[qt + 4 * i];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (j0 + 2 * kp + r <= p) total[r] += exp2f(fmaf(s[r][i], ksc[r], -off));
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        total[r] += __shfl_xor_sync(0xffffffffu, total[r], 1);
        total[r] += __shfl_xor_sync(0xffffffffu, total[r], 2);
        const int j = j0 + 2 * kp + r;
        if (qt || j >= base + live) continue;
        if (a.splits == 1)
            a.acc_out[seq0 + j] = a.acc_in ? fmaf(a.decay, a.acc_in[seq0 + j], total[r]) : total[r];
        else
            a.part[(static_cast<int64_t>(blockIdx.y) * a.batch + b) * a.max_ctx + j] = total[r];
    }
}

// The parts of a key's total, added in order.
__global__ void __launch_bounds__(256) accum_join_kernel(AccumArgs a, int blocks) {
    const int b = blockIdx.x / blocks;
    const int64_t j = static_cast<int64_t>(blockIdx.x - b * blocks) * 256 + threadIdx.x;
    const int live = live_rows(a.n_rows, b, a.n_q);
    if (j >= checked_base(a.q_pos0, b, live, a.max_ctx, a.status) + live) return;
    float t = 0.f;
    for (int s = 0; s < a.splits; ++s) t += a.part[(static_cast<int64_t>(s) * a.batch + b) * a.max_ctx + j];
    const int64_t at = static_cast<int64_t>(b) * a.cap + j;
    a.acc_out[at] = a.acc_in ? fmaf(a.decay, a.acc_in[at], t) : t;
}

template <typename TQ, typename TK, int D>
cudaError_t launch_simt(const AccumArgs& a, cudaStream_t st) {
    constexpr int smem = (S_KEYS + S_ROWS) * (D + 4) * 4;
    const cudaError_t e = cudaFuncSetAttribute(accum_simt_kernel<TQ, TK, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = static_cast<unsigned>((a.max_ctx + S_KEYS - 1) / S_KEYS);
    accum_simt_kernel<TQ, TK, D><<<dim3(tiles * a.batch, a.splits), 128, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

int plan_accum(int batch, int n_q, int heads, int kv_dtype, int64_t max_ctx) {
    const int64_t tiles = (max_ctx + S_KEYS - 1) / S_KEYS * batch;
    const int64_t rows = (static_cast<int64_t>(n_q) * heads + S_ROWS - 1) / S_ROWS;
    int64_t s = 3 * num_sms() / tiles;
    if (s > rows / 4) s = rows / 4;
    (void)kv_dtype;
    return s < 1 ? 1 : static_cast<int>(s);
}

size_t accum_ws_bytes(int batch, int splits, int64_t max_ctx) {
    return splits <= 1 ? 0 : sizeof(float) * static_cast<size_t>(splits) * batch * max_ctx;
}

cudaError_t launch_accum(const AccumArgs& a, cudaStream_t st) {
    cudaError_t e;
    const bool d128 = a.head_dim == 128;
    if (a.kv_dtype == HS2_F32) e = d128 ? launch_simt<float, float, 128>(a, st) : launch_simt<float, float, 64>(a, st);
    else if (a.kv_dtype == HS2_BF16)
        e = d128 ? launch_simt<__nv_bfloat16, __nv_bfloat16, 128>(a, st) : launch_simt<__nv_bfloat16, __nv_bfloat16, 64>(a, st);
    else e = d128 ? launch_simt<__nv_bfloat16, uint8_t, 128>(a, st) : launch_simt<__nv_bfloat16, uint8_t, 64>(a, st);
    if (e != cudaSuccess || a.splits == 1) return e;
    const int blocks = static_cast<int>((a.max_ctx + 255) / 256);
    accum_join_kernel<<<static_cast<unsigned>(blocks) * a.batch, 256, 0, st>>>(a, blocks);
    return cudaGetLastError();
}

}  // namespace hs2
