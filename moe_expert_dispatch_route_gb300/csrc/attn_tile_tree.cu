// attn_tile.cuh for rows that see the branch of a tree of drafted tokens that they stand on.
#include "attn_tile.cuh"

namespace moe {
namespace attn {

cudaError_t launch_tiles_tree(const moe_kv_cache& c, Params& p, int grid_cap, cudaStream_t st) {
    return launch_tiles_of<true>(c, p, grid_cap, st);
}

}  // namespace attn
}  // namespace moe
