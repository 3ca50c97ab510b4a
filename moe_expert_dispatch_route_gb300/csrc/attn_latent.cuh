// What the kernels of the absorbed latent attention share.
#pragma once

#include <cudaTypedefs.h>

#include "attn.cuh"

namespace moe {
namespace attn {

constexpr int kLatent = 512, kRope = 64, kWidth = kLatent + kRope;
constexpr int kSub = 64;                       // keys at a time
constexpr int kBlocks = kWidth / 64;           // 128-byte column blocks of a row
constexpr int kBlockBytes = kSub * 128;        // one of them
constexpr int kPieceBytes = 2 * kBlockBytes;   // 128 columns, as the second product takes them
constexpr int kPieces = kLatent / 128;

// A query tile's rows are (token, head), head fastest, p.group heads of a token.  A pair of CTAs (attn_latent_pair.cu)
// shares them out by heads where there are more than 64 (a tile is one token then), by tokens otherwise.
struct LatentParams {
    Params p;          // heads = 1
    int q_heads;       // of a token
    int cta_tokens;    // of a tile and CTA
    int split_heads;   // pairs: 1 by heads, 0 by tokens
};

// Key tiles of kSub keys of an item: [first, last), none for a tile that sees no key.
struct Subs {
    int first, last;
};
__device__ __forceinline__ Subs subs_of(const Item& it) {
    if (it.n == 0) return {0, 0};
    const int lo = max(it.s.lo, it.k0 * kKeyTile), hi = min(it.s.hi, (it.k0 + it.n) * kKeyTile);
    return {lo / kSub, (hi + kSub - 1) / kSub};
}

// What the second kernel has to know of a part, behind its sums in the workspace.  Every CTA writes those of
// its two slots in every call.
struct PartHead {
    int n;        // parts of the tile, 0: no part in this slot
    int rank;     // of this one among them
    int first;    // the CTA with the first one (in its slot 0; the others are in slot 1)
    int step;     // CTAs from one part to the next
    int rows;     // of the tile and CTA
    int token;    // its first row of q
    int head;     // and that row's head
};
__device__ __forceinline__ PartHead* part_head(const Params& p, int cta, int slot) {
    return reinterpret_cast<PartHead*>(part_ml(p, cta, slot) + 64);
}

// attn_latent_pair.cu: tiles of 65 to 128 rows, on pairs of CTAs
cudaError_t launch_latent_pair(const moe_latent_cache& c, const LatentParams& lp, int grid, cudaStream_t st);

// q as (d, head, token): a box holds a CTA's rows of a query tile.
bool make_latent_q_map(CUtensorMap* m, const LatentParams& lp);
// The pool as (d within a block, token, column block, page): a box holds `blocks` column blocks of `tokens` tokens.
bool make_latent_map(CUtensorMap* m, const moe_latent_cache& c, int blocks, int tokens);

}  // namespace attn
}  // namespace moe
