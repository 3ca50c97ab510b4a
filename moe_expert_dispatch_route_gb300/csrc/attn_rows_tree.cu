// attn_rows.cuh for rows that see the branch of a tree of drafted tokens that they stand on.
#include "attn_rows.cuh"

namespace moe {
namespace attn {

cudaError_t launch_rows_tree(const moe_kv_cache& c, Params& p, int rows, int grid_cap, cudaStream_t st) {
    return launch_rows_of<true>(c, p, rows, grid_cap, st);
}

}  // namespace attn
}  // namespace moe
