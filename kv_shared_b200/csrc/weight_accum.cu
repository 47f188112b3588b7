// weight_accum.cu -- accumulated attention weight of the cached keys: the fp32 kernel and
// the join of parts.
//
//   acc_out[j] = decay acc_in[j] + sum over rows r and heads h of
//                exp(scale q_rh . k_j - lse_rh)            [j <= p_r]
//
// The log-sum-exp is known, so one product S = K Q^T and one exponential per (key, row,
// head) are all there is; the keys stay put and the (row, head) pairs stream past, so that
// a key's total is a sum inside a thread and no key is read twice.
#include "common.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "window_keys.cuh"

namespace hs2 {
namespace {

constexpr int S_KEYS = 64;                       // keys per CTA

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

// fp32 caches on the CUDA cores.  Thread (kp, qt) of 32 x 4 has keys 2 kp, 2 kp + 1 and the PP
// pairs qt + 4 i of a tile (8; 4 where a sequence has no more than 16), two fp32 FMAs to an
// instruction.  Bound by the fp32 FMAs and the shared-memory loads between them (10 of 16 bytes to 64
// FMAs): 16 rows of 16 heads over 16000 keys of 128 52.9 us replayed on the same inputs (55.1 as a call
// among others), a single row over 131072 37.2.
template <int D, int PP>
__global__ void __launch_bounds__(128) accum_f32_kernel(AccumArgs a) {
    constexpr int S_ROWS = 4 * PP;               // (row, head) pairs per tile
    constexpr int LD = D + 4;
    extern __shared__ float4 sm4[];
    float* sk = reinterpret_cast<float*>(sm4);   // [64][LD]
    float* sq = sk + S_KEYS * LD;                // [S_ROWS][LD]
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
        const float4 x = j0 + r < base + live ? load4(static_cast<const float*>(a.k) + (seq0 + j0 + r) * D + 4 * c)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(sk + r * LD + 4 * c) = x;
    }
    float total[2] = {0.f, 0.f};
    for (int f0 = first; f0 < end; f0 += S_ROWS) {
        __syncthreads();
        for (int i = tid; i < S_ROWS * D / 4; i += 128) {
            const int r = i / (D / 4), c = i - r * (D / 4);
            const float4 x = f0 + r < end ? load4(static_cast<const float*>(a.q) + (flat0 + f0 + r) * D + 4 * c)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(sq + r * LD + 4 * c) = x;
        }
        if (tid < S_ROWS) {
            const int f = f0 + tid;
            s_lse[tid] = f < end ? a.lse[flat0 + f] * kLog2e : 0.f;
            s_pos[tid] = f < end ? base + f / a.heads : -1;
        }
        __syncthreads();
        float2 d[2][PP];                         // sums over the even and the odd dims
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < PP; ++i) d[r][i] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < D / 4; ++c) {
            const float4 x0 = *reinterpret_cast<const float4*>(sk + (2 * kp) * LD + 4 * c);
            const float4 x1 = *reinterpret_cast<const float4*>(sk + (2 * kp + 1) * LD + 4 * c);
#pragma unroll
            for (int i = 0; i < PP; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(sq + (qt + 4 * i) * LD + 4 * c);
                const float2 lo = make_float2(y.x, y.y), hi = make_float2(y.z, y.w);
                d[0][i] = fma2(make_float2(x0.x, x0.y), lo, fma2(make_float2(x0.z, x0.w), hi, d[0][i]));
                d[1][i] = fma2(make_float2(x1.x, x1.y), lo, fma2(make_float2(x1.z, x1.w), hi, d[1][i]));
            }
        }
        float s[2][PP];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < PP; ++i) s[r][i] = d[r][i].x + d[r][i].y;
#pragma unroll
        for (int i = 0; i < PP; ++i) {
            const int p = s_pos[qt + 4 * i];
            const float off = s_lse[qt + 4 * i];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (j0 + 2 * kp + r <= p) total[r] += exp2f(fmaf(s[r][i], sc2, -off));
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

template <int D, int PP>
cudaError_t launch_f32(const AccumArgs& a, cudaStream_t st) {
    constexpr int smem = (S_KEYS + 4 * PP) * (D + 4) * 4;
    const cudaError_t e = cudaFuncSetAttribute(accum_f32_kernel<D, PP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = static_cast<unsigned>((a.max_ctx + S_KEYS - 1) / S_KEYS);
    accum_f32_kernel<D, PP><<<dim3(tiles * a.batch, a.splits), 128, smem, st>>>(a);
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_f32(const AccumArgs& a, cudaStream_t st) {
    return static_cast<int64_t>(a.n_q) * a.heads <= 16 ? launch_f32<D, 4>(a, st) : launch_f32<D, 8>(a, st);
}

}  // namespace

int plan_accum(int batch, int n_q, int heads, int kv_dtype, int64_t max_ctx) {
    const bool f32 = kv_dtype == HS2_F32;
    const int64_t keys = f32 ? S_KEYS : 256, rows = f32 ? 32 : 128;
    const int64_t blocks = (max_ctx + keys - 1) / keys * batch, slots = (f32 ? 3 : 1) * num_sms();
    const int64_t tiles = (static_cast<int64_t>(n_q) * heads + rows - 1) / rows;
    // Parts of the pairs: the number that leaves the fewest idle SMs in the last round of key
    // blocks, each part with a few tiles of pairs; a part more has to save 1% (300 rows over 50000
    // bf16 keys, 196 blocks on 148 SMs: 118 us in one part, 84 in three).
    int best = 1;
    int64_t cost = -1;
    for (int64_t s = 1; s <= 64 && s * (f32 ? 4 : 2) <= (tiles > 1 ? tiles : 1) + (s == 1 ? 4 : 0); ++s) {
        const int64_t rounds = (blocks * s + slots - 1) / slots, c = rounds * 1000 / s + 10 * s;
        if (cost < 0 || c < cost) { cost = c; best = static_cast<int>(s); }
    }
    return best;
}

size_t accum_part_bytes(int batch, int splits, int64_t max_ctx) {
    const size_t n = splits <= 1 ? 0 : sizeof(float) * static_cast<size_t>(splits) * batch * max_ctx;
    return (n + 255) & ~static_cast<size_t>(255);
}

size_t accum_ws_bytes(int batch, int n_q, int heads, int head_dim, int kv_dtype, int splits, int64_t max_ctx) {
    const size_t q = kv_dtype == HS2_E4M3 ? static_cast<size_t>(batch) * n_q * heads * (2 * head_dim + sizeof(float)) : 0;
    return accum_part_bytes(batch, splits, max_ctx) + q;
}

cudaError_t launch_accum(const AccumArgs& a, cudaStream_t st) {
    const cudaError_t e = a.kv_dtype != HS2_F32 ? launch_accum_tile(a, st)
                                                : (a.head_dim == 128 ? launch_f32<128>(a, st) : launch_f32<64>(a, st));
    if (e != cudaSuccess || a.splits == 1) return e;
    const int blocks = static_cast<int>((a.max_ctx + 255) / 256);
    accum_join_kernel<<<static_cast<unsigned>(blocks) * a.batch, 256, 0, st>>>(a, blocks);
    return cudaGetLastError();
}

}  // namespace hs2
