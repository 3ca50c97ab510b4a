// attn_tile.cuh for rows that see the tokens before them.
#include "attn_tile.cuh"

namespace moe {
namespace attn {

cudaError_t launch_tiles(const moe_kv_cache& c, Params& p, int grid_cap, cudaStream_t st) {
    return launch_tiles_of<false>(c, p, grid_cap, st);
}

}  // namespace attn
}  // namespace moe
