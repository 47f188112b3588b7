// cache_ops_api.cu -- the extern "C" boundary of the calls around the block (declared in
// include/hs2.h): rows for the cache, sliding-window attention, accumulated attention
// weight, eviction.  Host code only: argument validation, workspace layout, dispatch.
#include <cmath>

#include "common.cuh"
#include "internal.h"

using namespace hs2;

namespace {

constexpr int64_t kIndexLimit = int64_t(1) << 31;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

struct Extent {
    const void* p;
    int64_t bytes;
};
bool overlap(const Extent& x, const Extent& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return x.p && y.p && (a <= b ? b - a < static_cast<uintptr_t>(x.bytes) : a - b < static_cast<uintptr_t>(y.bytes));
}

hs2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? HS2_OK : HS2_ERR_CUDA; }

// The fields that hs2_window_attn and hs2_weight_accum use.
hs2_status check_attn(const hs2_attn_desc* d) {
    if (!d) return HS2_ERR_INVALID_ARG;
    if (d->batch < 1 || d->n_q < 1 || d->heads < 1) return HS2_ERR_INVALID_ARG;
    if (d->kv_capacity < 1 || d->max_ctx < d->n_q || d->max_ctx > d->kv_capacity) return HS2_ERR_INVALID_ARG;
    if (!(d->softmax_scale >= 0.f) || std::isinf(d->softmax_scale)) return HS2_ERR_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 128) return HS2_ERR_UNSUPPORTED;
    if (d->heads > 128) return HS2_ERR_UNSUPPORTED;
    if (d->q_dtype == HS2_F32 ? d->kv_dtype != HS2_F32
                              : d->q_dtype != HS2_BF16 || (d->kv_dtype != HS2_BF16 && d->kv_dtype != HS2_E4M3))
        return HS2_ERR_UNSUPPORTED;
    if (d->kv_capacity >= kIndexLimit || d->batch * d->kv_capacity >= kIndexLimit) return HS2_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d->batch) * d->n_q * d->heads >= kIndexLimit) return HS2_ERR_UNSUPPORTED;
    return HS2_OK;
}

float eff_scale(const hs2_attn_desc* d) {
    return d->softmax_scale > 0.f ? d->softmax_scale : 1.f / std::sqrt(static_cast<float>(d->head_dim));
}

}  // namespace

extern "C" {

hs2_status hs2_qk_norm_rope(const hs2_rope_desc* desc, const void* q, const void* k, const void* v,
                            const float* q_weight, const float* k_weight, const double* inv_freq,
                            const int32_t* row0, const int32_t* pos, const int32_t* n_rows, void* q_out,
                            void* k_cache, void* v_cache, float* k_scale, float* v_scale, hs2_stream_t stream) {
    if (!desc || (!q && !k && !v) || !row0) return HS2_ERR_INVALID_ARG;
    const hs2_rope_desc& d = *desc;
    if (d.batch < 1 || d.n < 1 || d.heads < 1 || d.kv_capacity < 1) return HS2_ERR_INVALID_ARG;
    if (d.rot_dim < 0 || d.rot_dim > d.head_dim || !(d.eps >= 0.f) || std::isinf(d.eps)) return HS2_ERR_INVALID_ARG;
    if (d.head_dim != 64 && d.head_dim != 128) return HS2_ERR_UNSUPPORTED;
    if (d.rot_dim % 16 != 0 || d.heads > 128) return HS2_ERR_UNSUPPORTED;
    if (d.in_dtype != HS2_F32 && d.in_dtype != HS2_BF16) return HS2_ERR_UNSUPPORTED;
    if (d.kv_dtype != HS2_BF16 && d.kv_dtype != HS2_E4M3 && !(d.kv_dtype == HS2_F32 && d.in_dtype == HS2_F32))
        return HS2_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(d.batch) * d.n >= kIndexLimit || d.kv_capacity >= kIndexLimit ||
        d.batch * d.kv_capacity >= kIndexLimit || d.q_row >= kIndexLimit || d.k_row >= kIndexLimit ||
        d.v_row >= kIndexLimit)
        return HS2_ERR_UNSUPPORTED;
    const int per16 = d.in_dtype == HS2_F32 ? 4 : 8;
    const bool e4 = d.kv_dtype == HS2_E4M3;
    if (q && (!q_out || d.q_row < static_cast<int64_t>(d.heads) * d.head_dim || d.q_row % per16)) return HS2_ERR_INVALID_ARG;
    if (q && q == q_out && d.q_row != static_cast<int64_t>(d.heads) * d.head_dim) return HS2_ERR_INVALID_ARG;
    if (k && (!k_cache || d.k_row < d.head_dim || d.k_row % per16 || (e4 && !k_scale))) return HS2_ERR_INVALID_ARG;
    if (v && (!v_cache || d.v_row < d.head_dim || d.v_row % per16 || (e4 && !v_scale))) return HS2_ERR_INVALID_ARG;
    if (d.rot_dim > 0 && (q || k) && !inv_freq) return HS2_ERR_INVALID_ARG;
    const void* p16[] = {q, k, v, q_weight, k_weight, q_out, k_cache, v_cache, row0};
    for (const void* p : p16)
        if (!aligned16(p)) return HS2_ERR_INVALID_ARG;
    const void* p4[] = {k_scale, v_scale, pos, n_rows};
    for (const void* p : p4)
        if (!aligned4(p)) return HS2_ERR_INVALID_ARG;
    if (!aligned8(inv_freq)) return HS2_ERR_INVALID_ARG;
    RopeArgs a{};
    a.batch = d.batch; a.n = d.n; a.heads = d.heads; a.head_dim = d.head_dim;
    a.rot = inv_freq ? d.rot_dim : 0;
    a.interleaved = d.interleaved != 0; a.normalize = d.normalize != 0; a.in_f32 = d.in_dtype == HS2_F32;
    a.kv_dtype = d.kv_dtype; a.eps = d.eps; a.q_row = d.q_row; a.k_row = d.k_row; a.v_row = d.v_row;
    a.cap = d.kv_capacity; a.q = q; a.k = k; a.v = v; a.q_weight = q_weight; a.k_weight = k_weight;
    a.inv_freq = inv_freq; a.row0 = row0; a.pos = pos; a.n_rows = n_rows; a.q_out = q_out;
    a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    return from_cuda(launch_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hs2_window_workspace_size(const hs2_attn_desc* desc, int32_t sinks) {
    if (check_attn(desc) != HS2_OK || desc->window < 1 || sinks < 0) return 0;
    const WindowPlan p = plan_window(desc->batch, desc->n_q, desc->heads, desc->kv_dtype, desc->window, sinks,
                                     desc->max_ctx);
    return kStatusBytes + window_ws_bytes(desc->batch, desc->n_q, desc->heads, desc->head_dim, p);
}

hs2_status hs2_window_attn(const hs2_attn_desc* desc, int32_t sinks, const void* q, const void* k, const void* v,
                           const float* k_scale, const float* v_scale, const int32_t* q_pos0, const int32_t* n_rows,
                           void* o, float* lse, void* workspace, size_t ws_bytes, hs2_stream_t stream) {
    const hs2_status s = check_attn(desc);
    if (s != HS2_OK) return s;
    if (desc->window < 1 || sinks < 0) return HS2_ERR_INVALID_ARG;
    if (!q || !k || !v || !q_pos0 || !o || !workspace) return HS2_ERR_INVALID_ARG;
    if (desc->kv_dtype == HS2_E4M3 && (!k_scale || !v_scale)) return HS2_ERR_INVALID_ARG;
    const void* p16[] = {q, k, v, o, lse, q_pos0, workspace};
    for (const void* p : p16)
        if (!aligned16(p)) return HS2_ERR_INVALID_ARG;
    if (!aligned4(n_rows) || !aligned4(k_scale) || !aligned4(v_scale)) return HS2_ERR_INVALID_ARG;
    const WindowPlan plan = plan_window(desc->batch, desc->n_q, desc->heads, desc->kv_dtype, desc->window, sinks,
                                        desc->max_ctx);
    if (ws_bytes < kStatusBytes + window_ws_bytes(desc->batch, desc->n_q, desc->heads, desc->head_dim, plan))
        return HS2_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    WindowArgs a{};
    a.batch = desc->batch; a.n_q = desc->n_q; a.heads = desc->heads; a.head_dim = desc->head_dim;
    a.window = desc->window; a.sinks = sinks; a.cap = desc->kv_capacity; a.max_ctx = desc->max_ctx;
    a.q_pos0 = q_pos0; a.n_rows = n_rows; a.q = q; a.k = k; a.v = v;
    if (desc->kv_dtype == HS2_E4M3) { a.k_scale = k_scale; a.v_scale = v_scale; }
    a.kv_dtype = desc->kv_dtype; a.scale = eff_scale(desc); a.o = o; a.lse = lse;
    a.splits = plan.splits; a.status = reinterpret_cast<uint32_t*>(ws);
    const size_t flat = static_cast<size_t>(desc->batch) * desc->n_q * desc->heads;
    a.tile = plan.tile;
    a.wide = ws + kStatusBytes;
    a.wide_rows = plan.wide_rows;
    if (plan.splits > 1) {
        a.part_o = reinterpret_cast<float*>(ws + kStatusBytes + window_wide_bytes(desc->batch, desc->head_dim, plan));
        a.part_ml = reinterpret_cast<float2*>(a.part_o + flat * plan.splits * desc->head_dim);
    }
    return from_cuda(launch_window(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hs2_weight_accum_workspace_size(const hs2_attn_desc* desc) {
    if (check_attn(desc) != HS2_OK) return 0;
    const int splits = plan_accum(desc->batch, desc->n_q, desc->heads, desc->kv_dtype, desc->max_ctx);
    return kStatusBytes + accum_ws_bytes(desc->batch, desc->n_q, desc->heads, desc->head_dim, desc->kv_dtype, splits, desc->max_ctx);
}

hs2_status hs2_weight_accum(const hs2_attn_desc* desc, const void* q, const void* k, const float* k_scale,
                            const float* lse, const int32_t* q_pos0, const int32_t* n_rows, float decay,
                            const float* acc_in, float* acc_out, void* workspace, size_t ws_bytes,
                            hs2_stream_t stream) {
    const hs2_status s = check_attn(desc);
    if (s != HS2_OK) return s;
    if (!q || !k || !lse || !q_pos0 || !acc_out || !workspace) return HS2_ERR_INVALID_ARG;
    if (desc->kv_dtype == HS2_E4M3 && !k_scale) return HS2_ERR_INVALID_ARG;
    if (acc_in && (!(decay >= 0.f) || std::isinf(decay))) return HS2_ERR_INVALID_ARG;
    const void* p16[] = {q, k, lse, q_pos0, workspace};
    for (const void* p : p16)
        if (!aligned16(p)) return HS2_ERR_INVALID_ARG;
    if (!aligned4(n_rows) || !aligned4(k_scale) || !aligned4(acc_in) || !aligned4(acc_out)) return HS2_ERR_INVALID_ARG;
    const int splits = plan_accum(desc->batch, desc->n_q, desc->heads, desc->kv_dtype, desc->max_ctx);
    if (ws_bytes < kStatusBytes + accum_ws_bytes(desc->batch, desc->n_q, desc->heads, desc->head_dim, desc->kv_dtype, splits,
                                                 desc->max_ctx))
        return HS2_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    AccumArgs a{};
    a.batch = desc->batch; a.n_q = desc->n_q; a.heads = desc->heads; a.head_dim = desc->head_dim;
    a.cap = desc->kv_capacity; a.max_ctx = desc->max_ctx; a.q_pos0 = q_pos0; a.n_rows = n_rows; a.q = q; a.k = k;
    if (desc->kv_dtype == HS2_E4M3) a.k_scale = k_scale;
    a.kv_dtype = desc->kv_dtype; a.lse = lse; a.scale = eff_scale(desc); a.decay = decay;
    a.acc_in = acc_in; a.acc_out = acc_out; a.splits = splits;
    if (splits > 1) a.part = reinterpret_cast<float*>(ws + kStatusBytes);
    a.split_q = ws + kStatusBytes + accum_part_bytes(desc->batch, splits, desc->max_ctx);
    a.status = reinterpret_cast<uint32_t*>(ws);
    return from_cuda(launch_accum(a, reinterpret_cast<cudaStream_t>(stream)));
}

hs2_status hs2_kv_evict(const hs2_evict_desc* desc, const int32_t* len, const float* acc, const void* k,
                        const void* v, const float* k_scale, const float* v_scale, void* k_out, void* v_out,
                        float* k_scale_out, float* v_scale_out, float* acc_out, int32_t* idx, int32_t* new_len,
                        hs2_stream_t stream) {
    if (!desc || !len || !acc || !k || !v || !k_out || !v_out || !idx || !new_len) return HS2_ERR_INVALID_ARG;
    const hs2_evict_desc& d = *desc;
    if (d.batch < 1 || d.sinks < 0 || d.window < 0 || d.budget < 0 || d.kv_capacity < 1) return HS2_ERR_INVALID_ARG;
    const int64_t keep = static_cast<int64_t>(d.sinks) + d.window + d.budget;
    if (keep < 1 || d.out_capacity < keep) return HS2_ERR_INVALID_ARG;
    if (d.head_dim != 64 && d.head_dim != 128) return HS2_ERR_UNSUPPORTED;
    if (d.kv_dtype != HS2_F32 && d.kv_dtype != HS2_BF16 && d.kv_dtype != HS2_E4M3) return HS2_ERR_UNSUPPORTED;
    if (d.kv_capacity >= kIndexLimit || d.out_capacity >= kIndexLimit || d.batch * d.kv_capacity >= kIndexLimit ||
        d.batch * d.out_capacity >= kIndexLimit)
        return HS2_ERR_UNSUPPORTED;
    if (d.kv_dtype == HS2_E4M3 && (!k_scale || !v_scale || !k_scale_out || !v_scale_out)) return HS2_ERR_INVALID_ARG;
    const void* p16[] = {k, v, k_out, v_out};
    for (const void* p : p16)
        if (!aligned16(p)) return HS2_ERR_INVALID_ARG;
    const void* p4[] = {len, acc, acc_out, idx, new_len, k_scale, v_scale, k_scale_out, v_scale_out};
    for (const void* p : p4)
        if (!aligned4(p)) return HS2_ERR_INVALID_ARG;
    // the rows move in no order, so that a cache cannot be cut in place; the new lengths are written
    // when the lengths have been read and may take their place
    const bool e4 = d.kv_dtype == HS2_E4M3;
    const int64_t row = static_cast<int64_t>(d.head_dim) * (e4 ? 1 : d.kv_dtype == HS2_BF16 ? 2 : 4);
    const int64_t n_in = d.batch * d.kv_capacity, n_out = d.batch * d.out_capacity;
    const int64_t n_seq = static_cast<int64_t>(d.batch) * 4;
    const Extent in[] = {{len, n_seq}, {k, n_in * row}, {v, n_in * row}, {acc, n_in * 4},
                         {e4 ? k_scale : nullptr, n_in * 4}, {e4 ? v_scale : nullptr, n_in * 4}};
    const Extent out[] = {{new_len, n_seq}, {k_out, n_out * row}, {v_out, n_out * row}, {acc_out, n_out * 4},
                          {e4 ? k_scale_out : nullptr, n_out * 4}, {e4 ? v_scale_out : nullptr, n_out * 4},
                          {idx, d.batch * keep * 4}};
    for (const Extent& x : in)
        for (const Extent& y : out)
            if (overlap(x, y) && !(&x == in && &y == out && len == new_len)) return HS2_ERR_INVALID_ARG;
    // nor may outputs meet: k_out holds counts that the kept rows' places follow from
    for (const Extent& x : out)
        for (const Extent& y : out)
            if (&x < &y && overlap(x, y)) return HS2_ERR_INVALID_ARG;
    EvictArgs a{};
    a.batch = d.batch; a.head_dim = d.head_dim; a.kv_dtype = d.kv_dtype;
    a.sinks = d.sinks; a.window = d.window; a.budget = d.budget; a.cap = d.kv_capacity; a.out_cap = d.out_capacity;
    a.len = len; a.acc = acc; a.k = k; a.v = v; a.k_scale = k_scale; a.v_scale = v_scale;
    a.k_out = k_out; a.v_out = v_out; a.k_scale_out = k_scale_out; a.v_scale_out = v_scale_out;
    a.acc_out = acc_out; a.idx = idx; a.new_len = new_len;
    return from_cuda(launch_evict(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
