// C ABI of the serving operators: argument checks of the paged key/value cache, its attention
// and draft verification.  Every computing step runs in the kernels.
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "kernels.h"
#include "moe.h"

using namespace moe;

namespace moe {

bool rows_apart(int64_t T, int64_t H, int64_t ld, int64_t hs, int64_t width) {
    if ((T > 1 && ld < width) || (H > 1 && hs < width)) return false;
    if (T == 1 || H == 1) return true;
    if (ld - width >= (H - 1) * hs || hs - width >= (T - 1) * ld) return true;  // one inside the other
    // the tokens nearest to each head, before it and after it
    for (int64_t h = 1; h < H; ++h) {
        const int64_t t = h * hs / ld, past = h * hs - t * ld;
        if ((t < T && past < width) || (t + 1 < T && ld - past < width)) return false;
    }
    return true;
}

}  // namespace moe

namespace {

// A call without an SM budget may have more CTAs than fit at once where they are short and alike.
int grid_cap_any(int max_ctas) { return max_ctas > 0 ? max_ctas : INT32_MAX; }
int grid_cap_of(int max_ctas) { return max_ctas > 0 ? max_ctas : device_info().num_sms * 8; }

moe_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    if (getenv("MOE_DEBUG")) fprintf(stderr, "libmoe_gb300: CUDA error %s\n", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

moe_status check_cache(const moe_kv_cache* c) {
    if (!c || !c->k || !c->v || c->num_pages <= 0 || c->page_size <= 0 || c->num_heads <= 0 || c->head_dim <= 0)
        return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_BF16 && c->dtype != MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return MOE_ERR_UNSUPPORTED;
    if (c->page_size < 16 || (c->page_size & (c->page_size - 1))) return MOE_ERR_UNSUPPORTED;
    const bool fp8 = c->dtype == MOE_FP8_E4M3;
    if (fp8 != (c->k_scale != nullptr) || fp8 != (c->v_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (c->stride_page <= 0 || c->stride_head <= 0 || c->stride_token < c->head_dim) return MOE_ERR_INVALID_ARG;
    if (c->num_heads > 1 && c->stride_head < c->head_dim) return MOE_ERR_INVALID_ARG;
    const int64_t per16 = fp8 ? 16 : 8;  // elements in 16 bytes
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
        c->stride_page % per16 || c->stride_head % per16 || c->stride_token % per16)
        return MOE_ERR_ALIGNMENT;
    // byte strides of the copy engine's tensor maps are below 2^40
    const int64_t most = ((int64_t)1 << 40) / (fp8 ? 1 : 2);
    if (c->stride_page >= most || c->stride_head >= most || c->stride_token >= most) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status attn_paged(const moe_kv_cache* cache, const moe_attn_args* a, const uint64_t* tree, int32_t max_ctas,
                      moe_stream_t stream) {
    const moe_status s = check_cache(cache);
    if (s != MOE_OK) return s;
    if (!a || a->T < 0 || a->B < 0 || a->max_q < 0 || a->max_kv < 0 || a->table_ld < 0 || a->window < 0)
        return MOE_ERR_INVALID_ARG;
    if (a->num_q_heads <= 0 || a->num_q_heads % cache->num_heads || !isfinite(a->scale) || a->scale <= 0.0f)
        return MOE_ERR_INVALID_ARG;
    if (a->causal != 0 && a->causal != 1) return MOE_ERR_INVALID_ARG;
    if (a->num_q_heads / cache->num_heads > 64 || a->B > kMaxRequests) return MOE_ERR_UNSUPPORTED;
    if (a->T > kMaxTokens || a->max_kv > kMaxTokens) return MOE_ERR_UNSUPPORTED;
    if (a->T == 0 || a->B == 0 || a->max_q == 0) return MOE_OK;
    if (!a->q || !a->o || !a->cu_q || !a->kv_len || (a->table_ld > 0 && !a->block_table)) return MOE_ERR_INVALID_ARG;
    if (a->q_ld < 0 || a->q_head_stride < 0 || a->o_ld < 0 || a->o_head_stride < 0) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a->q) || !aligned16(a->o) || a->q_ld % 8 || a->q_head_stride % 8 || a->o_ld % 8 ||
        a->o_head_stride % 8)
        return MOE_ERR_ALIGNMENT;
    // no stride that is used reaches past a tensor map's (below 2^40 bytes) or what 64 bits count
    const int64_t T = a->T, H = a->num_q_heads, most = INT64_MAX / 2 / (T > H ? T : H), far = (int64_t)1 << 39;
    const int64_t limit = most < far ? most : far;
    if ((T > 1 && (a->q_ld >= limit || a->o_ld >= limit)) ||
        (H > 1 && (a->q_head_stride >= limit || a->o_head_stride >= limit)))
        return MOE_ERR_UNSUPPORTED;
    // rows of o that overlap would be written by several threads at once
    if (!rows_apart(T, H, a->o_ld, a->o_head_stride, cache->head_dim)) return MOE_ERR_INVALID_ARG;
    // work is counted in 31 bits: tiles of as few tokens as any kernel takes, against tiles of keys
    const int64_t group = a->num_q_heads / cache->num_heads, rows = a->max_q * group;
    const int64_t tokens = rows > kFewRows ? 128 / group * 2 : (rows <= 8 ? 8 : rows <= 16 ? 16 : 32) / group;
    if ((a->T / tokens + a->B) * cache->num_heads > INT32_MAX / ((int64_t)a->max_kv / 128 + 16))
        return MOE_ERR_UNSUPPORTED;
    if (!a->workspace || a->workspace_bytes < attn_workspace_bytes()) return MOE_ERR_WORKSPACE;
    if (!aligned_to(a->workspace, 256)) return MOE_ERR_ALIGNMENT;
    return cuda_status(launch_attn(*cache, *a, tree, grid_cap_of(max_ctas), (cudaStream_t)stream));
}

}  // namespace

extern "C" {

moe_status moe_kv_write(const moe_kv_cache* cache, int32_t T, const void* k, const void* v, int64_t ld_k, int64_t ld_v,
                        int64_t head_stride, const int64_t* slots, int32_t* err_flag, int32_t max_ctas,
                        moe_stream_t stream) {
    const moe_status s = check_cache(cache);
    if (s != MOE_OK) return s;
    if (T < 0 || (int64_t)T * 2 * cache->num_heads > ((int64_t)1 << 30)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!k || !v || !slots || ld_k < 0 || ld_v < 0 || head_stride < 0) return MOE_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned_to(slots, 8) || ld_k % 8 || ld_v % 8 || head_stride % 8)
        return MOE_ERR_ALIGNMENT;
    return cuda_status(launch_kv_write(*cache, T, k, v, ld_k, ld_v, head_stride, slots, err_flag,
                                       grid_cap_any(max_ctas), (cudaStream_t)stream));
}

moe_status moe_kv_read(const moe_kv_cache* cache, int32_t B, int32_t T, const int32_t* block_table, int32_t table_ld,
                       const int32_t* start, const int32_t* cu_len, void* k_out, void* v_out, int32_t* err_flag,
                       int32_t max_ctas, moe_stream_t stream) {
    const moe_status s = check_cache(cache);
    if (s != MOE_OK) return s;
    if (B < 0 || T < 0 || table_ld < 0) return MOE_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return MOE_OK;
    if (!block_table || !start || !cu_len || !k_out || !v_out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return MOE_ERR_ALIGNMENT;
    return cuda_status(launch_kv_read(*cache, B, T, block_table, table_ld, start, cu_len, k_out, v_out, err_flag,
                                      grid_cap_any(max_ctas), (cudaStream_t)stream));
}

size_t moe_attn_workspace_size(const moe_kv_cache* cache, int32_t num_q_heads) {
    if (check_cache(cache) != MOE_OK || num_q_heads <= 0 || num_q_heads % cache->num_heads) return 0;
    return attn_workspace_bytes();
}

moe_status moe_attn_paged(const moe_kv_cache* cache, const moe_attn_args* a, int32_t max_ctas, moe_stream_t stream) {
    return attn_paged(cache, a, nullptr, max_ctas, stream);
}

moe_status moe_attn_tree(const moe_kv_cache* cache, const moe_attn_args* a, const uint64_t* tree, int32_t max_ctas,
                         moe_stream_t stream) {
    if (a && a->T > 0 && !tree) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(tree, 8)) return MOE_ERR_ALIGNMENT;
    if (a && (a->causal != 1 || a->window != 0)) return MOE_ERR_INVALID_ARG;
    if (a && a->max_q > kMaxTree) return MOE_ERR_UNSUPPORTED;
    return attn_paged(cache, a, tree, max_ctas, stream);
}

moe_status moe_draft_verify(int32_t B, int32_t vocab, int32_t max_draft, int32_t dtype, const void* target,
                            int64_t target_ld, const void* draft, int64_t draft_ld, const int32_t* cu_draft,
                            const int32_t* ids, const float* u, const float* u_draw, int32_t* out_ids,
                            int32_t* out_len, int32_t* err_flag, int32_t max_ctas, moe_stream_t stream) {
    return moe_draft_verify_ex(B, INT32_MAX, vocab, max_draft, dtype, target, target_ld, draft, draft_ld, cu_draft, ids, u,
                               u_draw, out_ids, out_len, err_flag, max_ctas, stream);
}

moe_status moe_draft_verify_ex(int32_t B, int32_t N, int32_t vocab, int32_t max_draft, int32_t dtype, const void* target,
                               int64_t target_ld, const void* draft, int64_t draft_ld, const int32_t* cu_draft,
                               const int32_t* ids, const float* u, const float* u_draw, int32_t* out_ids,
                               int32_t* out_len, int32_t* err_flag, int32_t max_ctas, moe_stream_t stream) {
    if (B < 0 || N < 0 || vocab <= 0 || max_draft < 0 || target_ld < vocab || (draft && draft_ld < vocab))
        return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (vocab > (1 << 23) || max_draft > 255) return MOE_ERR_UNSUPPORTED;
    if (B == 0) return MOE_OK;
    if (!target || !cu_draft || !u_draw || !out_ids || !out_len) return MOE_ERR_INVALID_ARG;
    const uintptr_t el = dtype == MOE_F32 ? 4 : 2;
    if (!aligned_to(target, el) || !aligned_to(draft, el)) return MOE_ERR_ALIGNMENT;
    return cuda_status(launch_draft_verify(B, N, vocab, max_draft, dtype == MOE_F32, target, target_ld, draft, draft_ld,
                                           cu_draft, ids, u, u_draw, out_ids, out_len, err_flag,
                                           grid_cap_any(max_ctas), (cudaStream_t)stream));
}

}  // extern "C"
