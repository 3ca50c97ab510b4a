// moe_attn_paged, moe_attn_tree: picks the kernel for a call and builds its tensor maps.
#include "attn.cuh"

#include <cudaTypedefs.h>

namespace moe {
namespace attn {

bool make_pool_map(CUtensorMap* m, const moe_kv_cache& c, const void* base) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    const bool fp8 = c.dtype == MOE_FP8_E4M3;
    const cuuint64_t elt = fp8 ? 1 : 2;
    const cuuint32_t row = (cuuint32_t)(c.head_dim * elt < 128 ? c.head_dim * elt : 128);
    cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads,
                          (cuuint64_t)c.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)c.stride_token * elt, (cuuint64_t)c.stride_head * elt,
                             (cuuint64_t)c.stride_page * elt};
    cuuint32_t box[4] = {(cuuint32_t)(row / elt), (cuuint32_t)(c.page_size < kKeyTile ? c.page_size : kKeyTile), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn

size_t attn_workspace_bytes() {
    const size_t ctas = (size_t)device_info().num_sms;
    return attn::kMaxCtas * sizeof(uint32_t) + ctas * 2 * attn::kPartBytes;
}

cudaError_t launch_attn(const moe_kv_cache& c, const moe_attn_args& a, const uint64_t* tree, int grid_cap,
                        cudaStream_t st) {
    using namespace attn;
    Params p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.o = static_cast<uint16_t*>(a.o);
    p.lse = a.lse;
    p.q_ld = a.q_ld;
    p.q_head = a.q_head_stride;
    p.o_ld = a.o_ld;
    p.o_head = a.o_head_stride;
    p.cu_q = a.cu_q;
    p.kv_len = a.kv_len;
    p.table = a.block_table;
    p.table_ld = a.table_ld;
    p.T = a.T;
    p.B = a.B;
    p.max_q = a.max_q;
    p.max_kv = a.max_kv;
    p.heads = c.num_heads;
    p.group = a.num_q_heads / c.num_heads;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.page_shift = 0;
    while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.causal = tree ? 0 : a.causal;
    p.tree = tree;
    p.window = a.window < kMaxTokens ? a.window : kMaxTokens;  // no row is further from a token
    p.err = a.err_flag;
    p.counters = static_cast<uint32_t*>(a.workspace);
    p.parts = static_cast<uint8_t*>(a.workspace) + kMaxCtas * sizeof(uint32_t);
    p.inject_ns = wait_injection_ns();
    if (grid_cap > kMaxCtas) grid_cap = kMaxCtas;
    // Few rows are bound by reading the cache, on mma.sync; many on tcgen05, whose tiles have 128
    // rows whether they are filled or not.  32 requests of up to 8191 tokens, 8 heads of 128 (64),
    // bf16, rows a head: 32: 97 us against 113 there (63 against 96), 64: 161 against 113 (118
    // against 96); e4m3: 32: 129 against 147, 64: 189 against 148.  One rule for the whole call: one chunk of 512
    // tokens beside 127 single tokens takes 258 us here, 45 + 178 as two calls (e4m3: 354, 57 + 100).
    const int64_t rows = (int64_t)a.max_q * p.group;
    if (tree)
        return rows <= kFewRows ? launch_rows_tree(c, p, (int)rows, grid_cap, st) : launch_tiles_tree(c, p, grid_cap, st);
    return rows <= kFewRows ? launch_rows(c, p, (int)rows, grid_cap, st) : launch_tiles(c, p, grid_cap, st);
}

}  // namespace moe
