// C ABI of latent attention and of the norms around a block: argument checks.  Every computing step
// runs in the kernels.
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "kernels.h"
#include "moe.h"

using namespace moe;

namespace {

int grid_cap_any(int max_ctas) { return max_ctas > 0 ? max_ctas : INT32_MAX; }

moe_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    if (getenv("MOE_DEBUG")) fprintf(stderr, "libmoe_gb300: CUDA error %s\n", cudaGetErrorString(e));
    return MOE_ERR_CUDA;
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMostStride = (int64_t)1 << 39;  // in bf16 elements: a tensor map's strides are below 2^40 bytes

// A stride that is used (more than one of its index): no tensor map's limit, nor what 64 bits count, is passed.
bool stride_ok(int64_t stride, int64_t count, int64_t other) {
    const int64_t most = INT64_MAX / 2 / (count > other ? count : other);
    return count <= 1 || stride < (most < kMostStride ? most : kMostStride);
}

moe_status check_latent(const moe_latent_cache* c) {
    if (!c || !c->kv || c->num_pages <= 0 || c->page_size <= 0 || c->latent <= 0 || c->rope <= 0)
        return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_BF16 || c->latent != 512 || c->rope != 64) return MOE_ERR_UNSUPPORTED;
    if (c->page_size < 16 || (c->page_size & (c->page_size - 1))) return MOE_ERR_UNSUPPORTED;
    if (c->stride_page <= 0 || c->stride_token < c->latent + c->rope) return MOE_ERR_INVALID_ARG;
    if (!aligned16(c->kv) || c->stride_page % 8 || c->stride_token % 8) return MOE_ERR_ALIGNMENT;
    if (c->stride_page >= kMostStride || c->stride_token >= kMostStride) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_latent_write(const moe_latent_cache* cache, int32_t T, const void* c, int64_t ld_c, const void* k_rope,
                            int64_t ld_rope, const void* weight, float eps, const int64_t* slots, int32_t* err_flag,
                            int32_t max_ctas, moe_stream_t stream) {
    const moe_status s = check_latent(cache);
    if (s != MOE_OK) return s;
    if (T < 0 || !(eps >= 0.0f) || !isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!c || !k_rope || !slots || ld_c < 0 || ld_rope < 0) return MOE_ERR_INVALID_ARG;
    if (!aligned16(c) || !aligned16(k_rope) || !aligned16(weight) || !aligned_to(slots, 8) || ld_c % 8 || ld_rope % 8)
        return MOE_ERR_ALIGNMENT;
    if (!stride_ok(ld_c, T, 1) || !stride_ok(ld_rope, T, 1)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(launch_latent_write(*cache, T, c, ld_c, k_rope, ld_rope, weight, eps, slots, err_flag,
                                           grid_cap_any(max_ctas), (cudaStream_t)stream));
}

size_t moe_attn_latent_workspace_size(const moe_latent_cache* cache, int32_t num_q_heads) {
    if (check_latent(cache) != MOE_OK || num_q_heads <= 0 || num_q_heads > kMaxLatentHeads) return 0;
    return attn_workspace_bytes();
}

moe_status moe_attn_latent(const moe_latent_cache* cache, const moe_attn_args* a, const uint64_t* tree,
                           int32_t max_ctas, moe_stream_t stream) {
    const moe_status s = check_latent(cache);
    if (s != MOE_OK) return s;
    if (!a || a->T < 0 || a->B < 0 || a->max_q < 0 || a->max_kv < 0 || a->table_ld < 0 || a->window < 0)
        return MOE_ERR_INVALID_ARG;
    if (a->num_q_heads <= 0 || !isfinite(a->scale) || a->scale <= 0.0f) return MOE_ERR_INVALID_ARG;
    if (a->causal != 0 && a->causal != 1) return MOE_ERR_INVALID_ARG;
    if (tree && (a->causal != 1 || a->window != 0)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(tree, 8)) return MOE_ERR_ALIGNMENT;
    if (a->num_q_heads > kMaxLatentHeads || a->B > kMaxRequests || (tree && a->max_q > kMaxTree))
        return MOE_ERR_UNSUPPORTED;
    if (a->T > kMaxTokens || a->max_kv > kMaxTokens) return MOE_ERR_UNSUPPORTED;
    if (a->T == 0 || a->B == 0 || a->max_q == 0) return MOE_OK;
    if (!a->q || !a->o || !a->cu_q || !a->kv_len || (a->table_ld > 0 && !a->block_table)) return MOE_ERR_INVALID_ARG;
    if (a->q_ld < 0 || a->q_head_stride < 0 || a->o_ld < 0 || a->o_head_stride < 0) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a->q) || !aligned16(a->o) || a->q_ld % 8 || a->q_head_stride % 8 || a->o_ld % 8 ||
        a->o_head_stride % 8)
        return MOE_ERR_ALIGNMENT;
    const int64_t T = a->T, H = a->num_q_heads;
    if (!stride_ok(a->q_ld, T, H) || !stride_ok(a->o_ld, T, H) || !stride_ok(a->q_head_stride, H, T) ||
        !stride_ok(a->o_head_stride, H, T))
        return MOE_ERR_UNSUPPORTED;
    // rows of o that overlap would be written by several threads at once
    if (!rows_apart(T, H, a->o_ld, a->o_head_stride, cache->latent)) return MOE_ERR_INVALID_ARG;
    // work is counted in 31 bits: query tiles of at least one token against tiles of keys
    const int64_t group = H > 64 ? (H + 1) / 2 : H, most = 64 / group, per_tile = a->max_q < most ? a->max_q : most;
    if (T / per_tile + a->B > INT32_MAX / ((int64_t)a->max_kv / 128 + 16)) return MOE_ERR_UNSUPPORTED;
    if (!a->workspace || a->workspace_bytes < attn_workspace_bytes()) return MOE_ERR_WORKSPACE;
    if (!aligned_to(a->workspace, 256)) return MOE_ERR_ALIGNMENT;
    return cuda_status(launch_attn_latent(*cache, *a, tree, grid_cap_any(max_ctas), (cudaStream_t)stream));
}

size_t moe_attn_expanded_workspace_size(int32_t num_heads) { return num_heads > 0 ? attn_workspace_bytes() : 0; }

moe_status moe_attn_expanded(const moe_attn_expanded_args* a, int32_t max_ctas, moe_stream_t stream) {
    if (!a || a->T < 0 || a->S < 0 || a->B < 0 || a->max_q < 0 || a->max_kv < 0) return MOE_ERR_INVALID_ARG;
    if (a->num_heads <= 0 || !isfinite(a->scale) || a->scale <= 0.0f) return MOE_ERR_INVALID_ARG;
    if (a->causal != 0 && a->causal != 1) return MOE_ERR_INVALID_ARG;
    if (a->num_heads > 4096 || a->B > kMaxRequests || a->T > kMaxTokens || a->S > kMaxTokens || a->max_kv > kMaxTokens)
        return MOE_ERR_UNSUPPORTED;
    if (a->T == 0 || a->B == 0 || a->max_q == 0) return MOE_OK;
    if (!a->q || !a->o || !a->cu_q || !a->cu_kv || (a->S > 0 && (!a->k || !a->k_rope || !a->v)))
        return MOE_ERR_INVALID_ARG;
    const int64_t strides[] = {a->q_ld, a->q_head_stride, a->k_ld, a->k_head_stride, a->rope_ld,
                               a->v_ld, a->v_head_stride, a->o_ld, a->o_head_stride};
    for (int64_t x : strides)
        if (x < 0) return MOE_ERR_INVALID_ARG;
    for (int64_t x : strides)
        if (x % 8) return MOE_ERR_ALIGNMENT;
    if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->k_rope) || !aligned16(a->v) || !aligned16(a->o))
        return MOE_ERR_ALIGNMENT;
    const int64_t T = a->T, S = a->S, H = a->num_heads;
    if (!stride_ok(a->q_ld, T, H) || !stride_ok(a->o_ld, T, H) || !stride_ok(a->k_ld, S, H) || !stride_ok(a->v_ld, S, H) ||
        !stride_ok(a->rope_ld, S, 1) || !stride_ok(a->q_head_stride, H, T) || !stride_ok(a->o_head_stride, H, T) ||
        !stride_ok(a->k_head_stride, H, S) || !stride_ok(a->v_head_stride, H, S))
        return MOE_ERR_UNSUPPORTED;
    if (!rows_apart(T, H, a->o_ld, a->o_head_stride, 128)) return MOE_ERR_INVALID_ARG;
    // work is counted in 31 bits: query tiles of 256 rows of a head against tiles of keys
    if ((T / 256 + a->B) * H > INT32_MAX / ((int64_t)a->max_kv / 128 + 16)) return MOE_ERR_UNSUPPORTED;
    if (!a->workspace || a->workspace_bytes < attn_workspace_bytes()) return MOE_ERR_WORKSPACE;
    if (!aligned_to(a->workspace, 256)) return MOE_ERR_ALIGNMENT;
    return cuda_status(launch_attn_expanded(*a, grid_cap_any(max_ctas), (cudaStream_t)stream));
}

moe_status moe_block_norm(const moe_norm_args* a, int32_t max_ctas, moe_stream_t stream) {
    if (!a || a->T < 0 || a->hidden <= 0) return MOE_ERR_INVALID_ARG;
    if ((a->dtype != MOE_F32 && a->dtype != MOE_BF16) || (a->resid_dtype != MOE_F32 && a->resid_dtype != MOE_BF16))
        return MOE_ERR_UNSUPPORTED;
    if (a->hidden % 8 || a->hidden > kMaxNormWidth) return MOE_ERR_UNSUPPORTED;
    if (!isfinite(a->scale) || !(a->eps >= 0.0f) || !isfinite(a->eps)) return MOE_ERR_INVALID_ARG;
    if (a->T == 0) return MOE_OK;
    if (!a->y || (!a->out && !a->resid_out) || (a->out && !a->pre_weight)) return MOE_ERR_INVALID_ARG;
    if (a->gate && a->gate_rows != 1 && a->gate_rows != a->T) return MOE_ERR_INVALID_ARG;
    const void* all[] = {a->y, a->post_weight, a->gate, a->resid, a->resid_out, a->pre_weight, a->out};
    for (const void* x : all)
        if (!aligned16(x)) return MOE_ERR_ALIGNMENT;
    return cuda_status(launch_block_norm(*a, grid_cap_any(max_ctas), (cudaStream_t)stream));
}

}  // extern "C"
