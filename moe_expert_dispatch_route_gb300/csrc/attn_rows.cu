// attn_rows.cuh for rows that see the tokens before them.
#include "attn_rows.cuh"

namespace moe {
namespace attn {

cudaError_t launch_rows(const moe_kv_cache& c, Params& p, int rows, int grid_cap, cudaStream_t st) {
    return launch_rows_of<false>(c, p, rows, grid_cap, st);
}

}  // namespace attn
}  // namespace moe
