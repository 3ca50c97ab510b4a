// Latent attention, absorbed form, for requests of more than 64 rows: a query tile of up to 128 rows, half of
// them (of a token's heads, or of the tokens) in each CTA of a pair (a cluster of two), over the same range of
// keys, 64 at a time.  The pair's MMAs (cta_group::2) read each operand from where it lies:
//   S = Q K^T    m = 128 rows, n = 64 keys, k = 576     each CTA holds its 64 rows of Q and 32 of the keys
//   O += P V     m = 128 rows, n = 2 x 256 columns, k = 64 keys     its rows of P and half of the columns
// so that a CTA copies 68 KB for 64 keys where each of two single CTAs copies 72, and its tensor cores read two
// thirds of what theirs do: shared memory bounds those (64 requests of up to 16384 tokens with 128 heads: 201 us on
// single CTAs side by side, 150 here; two chunks of 64 tokens over 8192 256 and 150).  An accumulator of 64 rows a CTA
// fills all 128 lanes: lanes 0-63 hold the first half of its columns, lanes 64-127 the second.  A row is thus shared
// by two threads, here for half of the keys' scores and half of the output's columns each, and everything but the
// MMAs' operands stays in its CTA.
//
// What bounds it now: 2370 cycles for 64 keys, of which the MMAs last 1100 and a softmax 1100; the scores wait for
// keys, which come about 3000 cycles after they are asked for, and with Q beside them two stages fill shared memory (HBM
// alone would take 1570; tensor memory has 192 columns left, which are not used).  Three stages with one of values 222 us, keys in thirds 152-168, tiles fetched into L2
// ahead of time 175.
//
// The running maximum is followed loosely, as in attn_tile.cuh.  Split tiles are joined by attn_latent.cu's
// second kernel.
//
//   warps 0-3   softmax, rescaling and epilogue: warps w and w + 2 share the rows 32 w ..
//   warp 4      the scores' MMAs (first CTA); tells it that scores have been read (the other)
//   warp 5      values: zeros what no row sees; the products' MMAs (first CTA); tells it that values and
//               probabilities are there (the other)
//   warps 6, 7  copies of Q and keys; of values
//
// The first CTA's barriers count both CTAs' arrivals and copies; its commits reach both.
#include "attn_latent.cuh"

namespace moe {
namespace tc {

// Tiled loads into this CTA's shared memory, signalled on the mbarrier at cluster address `bar`.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                                 int c3, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}
// Arrives on an mbarrier of another CTA of the cluster, ordered after what this CTA has done, at its own scope: what
// is told is that this SM's tensor core may read this CTA's shared memory (its writers' proxy fences come
// before), or write its tensor memory.  No thread of the other CTA reads any of it.  PTX's memory model does not
// cover that: a release at this scope orders nothing for a thread of the other CTA, the one that issues the MMA.  That the
// reader is the writers' own SM, whose shared memory holds what they have fenced, is a property of this chip (sm_103a),
// which is all this file is compiled for.  (Released at cluster scope, an arrival took 1900 cycles to be seen, on the
// chain that bounds the kernel: 210 us where this takes 150.)
__device__ __forceinline__ void mbar_tell_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// mbar_wait for phases that threads of the other CTA complete too.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((n & 63u) == 0) {
            if (*abort) return false;
            const uint64_t now = globaltimer();
            if (t0 == 0) t0 = now;
            else if (now - t0 > kWaitTimeoutNs) return false;
        }
    }
}

}  // namespace tc

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;                       // of a CTA
constexpr int kStages = 2;                      // of keys, and of values
constexpr int kQBytes = kBlocks * kRows * 128;
constexpr int kPBytes = kRows * 128;
constexpr int kKeyBlock = kSub / 2 * 128;       // 64 columns of a CTA's keys
constexpr int kKeyBytes = kBlocks * kKeyBlock;
constexpr int kValueBytes = 2 * kPieceBytes;    // a CTA's columns: 128 of each half of 256
constexpr int kBars = 5 * kStages + 2 + 2 + 2 + 2 + 2 + 2;
constexpr int kTail = kBars * 8 + 16 + 4 * kRows * 4;
constexpr int kSmem = 1024 + kQBytes + kPBytes + kStages * (kKeyBytes + kValueBytes) + kTail;
static_assert(kSmem <= 232448 - 512, "");
static_assert(kStages * (kKeyBytes + kValueBytes) >= (kMaxRequests + 32) * 4, "locate()'s scratch");
static_assert(kKeyBytes % 1024 == 0, "swizzled tiles");

// What the scores' warp has to know of a key tile, put beside it by the copying warp.
enum : uint32_t {
    kNewQ = 1u,  // the first one of a query tile
    kLast = 2u,  // the last one
    kStop = 4u   // no more
};

template <bool kTree>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    attn_latent_pair_kernel(const __grid_constant__ LatentParams lp, const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    const Params& p = lp.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* qs = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);  // by an offset: accesses keep 32-bit addresses
    uint8_t* ps = qs + kQBytes;
    uint8_t* keys = ps + kPBytes;
    uint8_t* vals = keys + kStages * kKeyBytes;
    uint64_t* k_full = reinterpret_cast<uint64_t*>(vals + kStages * kValueBytes);  // first CTA: of both CTAs' keys
    uint64_t* k_empty = k_full + kStages;
    uint64_t* v_full = k_empty + kStages;  // of this CTA's values
    uint64_t* v_peer = v_full + kStages;   // first CTA: the other one's are there, and its probabilities
    uint64_t* v_empty = v_peer + kStages;
    uint64_t* s_full = v_empty + kStages;  // [2]
    uint64_t* s_free = s_full + 2;         // [2] the scores have been read (first CTA: by both)
    uint64_t* q_full = s_free + 2;         // first CTA: of both
    uint64_t* q_empty = q_full + 1;
    uint64_t* p_full = q_empty + 1;        // this CTA's probabilities
    uint64_t* pv_done = p_full + 1;
    uint64_t* done = pv_done + 1;
    uint64_t* never = done + 1;
    uint32_t* cmds = reinterpret_cast<uint32_t*>(never + 1);     // [kStages]
    float* row_max = reinterpret_cast<float*>(cmds + 4);         // [2][kRows] of each half of the keys
    float* row_sum = row_max + 2 * kRows;                        // likewise
    __shared__ Start start;
    __shared__ int abort_s;
    __shared__ uint32_t tmem_s;
    volatile int* abort = &abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int me = blockIdx.x >> 1, block = (int)tc::cluster_rank();
    const bool first_cta = block == 0;
    constexpr int kMmaWarp = 4, kValueWarp = 5, kKeyCopies = 6, kValueCopies = 7;
    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&k_full[i], 1);
            tc::mbar_init(&k_empty[i], 1);
            tc::mbar_init(&v_full[i], 1);
            tc::mbar_init(&v_peer[i], 1);
            tc::mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s_full[i], 1);
            tc::mbar_init(&s_free[i], first_cta ? 5 : 4);
        }
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_empty, 1);
        tc::mbar_init(p_full, 4);
        tc::mbar_init(pv_done, 1);
        tc::mbar_init(done, 1);
        tc::mbar_init(never, 1);
        tc::fence_barrier_init();
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    // both CTAs' barriers are there before any remote arrival or copy, and both run before the pair allocates
    tc::cluster_sync();
    pdl_begin();
    if (warp == kMmaWarp) {
        tc::tmem_alloc_pair(&tmem_s, 512);
        tc::tmem_relinquish_pair();
        tc::tc_fence_before();
    }
    locate<kThreads>(p, reinterpret_cast<uint32_t*>(keys), &start, me, gridDim.x >> 1);
    tc::tc_fence_after();
    const uint32_t tmem = tmem_s;
    if (threadIdx.x < 2) part_head(p, blockIdx.x, threadIdx.x)->n = 0;
    __syncthreads();
    if (p.inject_ns > 0 && me == 0) {  // test hook: the failure path of a bounded wait
        if (threadIdx.x == 0) {
            tc::wait_on_nothing(never, (uint64_t)p.inject_ns);
            set_err(p.err, MOE_ERR_TIMEOUT);
        }
        __syncthreads();
        tc::cluster_sync();
        if (warp == kMmaWarp) tc::tmem_dealloc_pair(tmem, 512);
        return;
    }
    Cursor cur = cursor(start);
    // a wait that runs out is reported and then passed, here and in every later wait, so that
    // each barrier is still met; the results are void
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!tc::mbar_wait(bar, parity, abort)) {
            set_err(p.err, MOE_ERR_TIMEOUT);
            *abort = 1;
        }
    };
    auto wait_both = [&](uint64_t* bar, uint32_t parity) {
        if (!tc::mbar_wait_cluster(bar, parity, abort)) {
            set_err(p.err, MOE_ERR_TIMEOUT);
            *abort = 1;
        }
    };
    // this CTA's part of a query tile
    const int head0 = lp.split_heads ? block * p.group : 0, token0 = lp.split_heads ? 0 : block * lp.cta_tokens;
    constexpr uint32_t kScores = 256;  // column of the score buffers, 32 each, behind the output's two of 128

    if (warp == kKeyCopies || warp == kValueCopies) {
        // ------------------------------------------------------------ copies
        const bool is_k = warp == kKeyCopies;
        // several query tiles read the same keys, one leaves L2 to the parts of split tiles (two chunks of 64
        // tokens with 128 heads: 151 us, 173 if their keys gave way)
        const uint64_t policy = tc::policy_of(p.max_q <= p.tokens_per_tile);
        const int span_keys = is_k ? kSub / 2 : kSub;             // of a tile that this CTA copies
        const int box_keys = min(p.page_size, span_keys), npg = span_keys / box_keys;
        const int blks = is_k ? kBlocks : 4;                      // column blocks
        const int per_box = npg == 1 ? (is_k ? kBlocks : 2) : 1;  // of them in a copy
        const int per_page = blks / per_box;                      // copies
        uint64_t* full = is_k ? k_full : v_full;
        uint64_t* empty = is_k ? k_empty : v_empty;
        uint32_t tiles = 0, sent = 0, items = 0, q_sent = 0;
        bool more_now = more(cur);
        Item it, after;
        Pages pages, pages_after;
        if (more_now) {
            it = take(p, cur);
            pages = pages_of(p, it);
        }
        for (; more_now; it = after, pages = pages_after) {
            auto ahead = [&] {  // the next query tile's lengths and first table entries
                more_now = more(cur);
                if (more_now) {
                    after = take(p, cur);
                    pages_after = pages_of(p, after);
                }
            };
            const Subs s = subs_of(it);
            if (s.first >= s.last) {
                ahead();
                continue;
            }
            if (is_k) {
                if (items > 0) wait(q_empty, (items - 1) & 1);
                ++items;
                if (!*abort) {
                    ++q_sent;
                    if (first_cta && lane == 0) tc::mbar_arrive_expect_tx(q_full, 2 * kBlocks * lp.cta_tokens * p.group * 128);
                    __syncwarp();
                    if (lane < kBlocks)
                        tc::tma_load_3d_pair(qs + lane * kRows * 128, &qmap, tc::map_to_rank(q_full, 0), lane * 64, head0,
                                             it.r.row0 + it.tile * p.tokens_per_tile + token0);
                }
            }
            for (int k = s.first; k < s.last; ++k, ++tiles) {
                const int key0 = k * kSub, mine0 = key0 + (is_k ? block * (kSub / 2) : 0);
                const uint32_t st = tiles % kStages, turn = tiles / kStages;
                // lane i: copy i % per_page of page i / per_page of this CTA's keys
                const int pg = lane / per_page, part = lane % per_page;
                auto seen = [&](int key) { return key < it.s.hi && key + box_keys > it.s.lo; };
                const int key = mine0 + pg * box_keys, off = key & (p.page_size - 1);
                const bool want = pg < npg && seen(key);
                int page = page_of(p, it, pages, key0, (key >> p.page_shift) - (key0 >> p.page_shift));
                if (want && (page < 0 || page >= p.num_pages)) {
                    set_err(p.err, MOE_ERR_BAD_INDEX);
                    page = p.num_pages;  // past the pool: the copy fills zeros
                }
                if (turn > 0) wait(&empty[st], (turn - 1) & 1);
                if (is_k && first_cta && lane == 0)
                    cmds[st] = (k == s.first ? kNewQ : 0) | (k == s.last - 1 ? kLast : 0);
                if (k == s.first) ahead();
                if (*abort) continue;
                sent = tiles + 1;
                // keys are signalled to the first CTA, which announces both CTAs' bytes
                uint32_t bytes = __popc(__ballot_sync(0xffffffffu, want)) * per_box * box_keys * 128;
                if (is_k) {
                    const int other = mine0 + kSub / 2;
                    for (int i = 0; i < npg; ++i)
                        if (seen(other + i * box_keys)) bytes += kBlocks * box_keys * 128;
                }
                if ((!is_k || first_cta) && lane == 0) tc::mbar_arrive_expect_tx(&full[st], bytes);
                __syncwarp();
                if (want) {
                    if (is_k)
                        tc::tma_load_4d_pair(keys + st * kKeyBytes + part * kKeyBlock + pg * box_keys * 128, &kmap,
                                             tc::map_to_rank(&full[st], 0), 0, off, part * per_box, page, policy);
                    else {
                        // this CTA's blocks: 2 and 2 of the two halves of 256 columns
                        const int blk = part * per_box;
                        tc::tma_load_4d_hint(vals + st * kValueBytes + blk * kBlockBytes + pg * box_keys * 128, &vmap,
                                             &full[st], 0, off, (blk >> 1) * 4 + block * 2 + (blk & 1), page, policy);
                    }
                }
            }
        }
        if (*abort) {  // copies still in flight land (or a bounded wait gives up) before the CTA ends
            if (is_k && !first_cta) {  // signalled to the other CTA: a time far above any copy's
                const uint64_t t0 = tc::globaltimer();
                while (tc::globaltimer() - t0 < 2000000ull) {
                }
            } else {
                for (uint32_t t = sent, i = 0; t-- > 0 && i < kStages; ++i)
                    tc::mbar_wait_bounded(&full[t % kStages], t / kStages & 1);
                if (q_sent > 0) tc::mbar_wait_bounded(q_full, (q_sent - 1) & 1);
            }
        }
        if (is_k && first_cta) {
            const uint32_t st = tiles % kStages, turn = tiles / kStages;
            if (turn > 0) wait(&empty[st], (turn - 1) & 1);
            if (lane == 0) {
                cmds[st] = kStop;
                tc::mbar_arrive(&full[st]);
            }
        }
    } else if (warp == kMmaWarp) {
        if (first_cta) {
            // -------------------------------------------------------- the scores' MMAs
            constexpr uint32_t kIdescS = tc::idesc_bf16_f32(128, kSub);
            uint32_t tiles = 0, queries = 0;
            const uint64_t q_desc = tc::desc_sw128_kmajor(tc::smem_u32(qs));
            const uint64_t k_desc = tc::desc_sw128_kmajor(tc::smem_u32(keys));
            for (;; ++tiles) {
                const uint32_t st = tiles % kStages;
                wait(&k_full[st], tiles / kStages & 1);
                const uint32_t cmd = cmds[st];
                if (cmd & kStop) break;
                if (cmd & kNewQ) wait(q_full, queries++ & 1);
                if (tiles > 1) wait_both(&s_free[tiles & 1], (tiles >> 1) - 1 & 1);  // the buffer's scores have been read
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    const uint64_t b = k_desc + st * (kKeyBytes >> 4);
                    const uint32_t to = tmem + kScores + (tiles & 1) * (kSub / 2);
#pragma unroll
                    for (int s = 0; s < kWidth / 16; ++s)
                        tc::mma_bf16_pair(to, q_desc + (s / 4) * (kRows * 128 >> 4) + s % 4 * 2,
                                          b + (s / 4) * (kKeyBlock >> 4) + s % 4 * 2, kIdescS, s > 0);
                    tc::mma_commit_pair(&k_empty[st], 3);
                    tc::mma_commit_pair(&s_full[tiles & 1], 3);
                    if (cmd & kLast) tc::mma_commit_pair(q_empty, 3);
                }
                __syncwarp();
            }
            if (tc::elect_one()) tc::mma_commit_pair(done, 3);
            __syncwarp();
        } else {
            // tells the first CTA that the scores have been read: from the softmax's warps, the remote arrivals took
            // 1500 cycles a tile
            uint32_t n = 0;
            while (more(cur)) {
                const Item it = take(p, cur);
                const Subs s = subs_of(it);
                for (int k = s.first; k < s.last; ++k, ++n) {
                    wait(&s_free[n & 1], n >> 1 & 1);
                    if (lane == 0) tc::mbar_tell_remote(tc::map_to_rank(&s_free[n & 1], 0));
                }
            }
        }
        tc::mbar_wait_bounded(done, 0);
    } else if (warp == kValueWarp) {
        // ------------------------------------------------------------ values, and the products' MMAs
        constexpr uint32_t kIdescO = tc::idesc_bf16_f32(128, 256) | kIdescBMn;
        const uint64_t p_desc = tc::desc_sw128_kmajor(tc::smem_u32(ps));
        const uint64_t v_desc = desc_sw128_mnmajor(tc::smem_u32(vals), kBlockBytes);
        uint32_t n = 0;  // key tiles so far
        while (more(cur)) {
            const Item it = take(p, cur);
            const Subs s = subs_of(it);
            for (int k = s.first; k < s.last; ++k, ++n) {
                const uint32_t st = n % kStages, turn = n / kStages;
                wait(&v_full[st], turn & 1);
                const int z0 = it.s.lo - k * kSub, z1 = it.s.hi - k * kSub;
                if (z0 > 0 || z1 < kSub) {
                    // keys that no row sees hold anything, NaN among it: 0 * NaN would reach o
                    uint4* row = reinterpret_cast<uint4*>(vals + st * kValueBytes);
                    for (int i = lane; i < kSub * 32; i += 32) {
                        const int r = (i >> 3) & (kSub - 1);
                        if (r < z0 || r >= z1) row[i] = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                wait(p_full, n & 1);
                if (!first_cta) {
                    if (lane == 0) tc::mbar_tell_remote(tc::map_to_rank(&v_peer[st], 0));
                    continue;
                }
                wait_both(&v_peer[st], turn & 1);
                tc::tc_fence_after();
                const uint32_t accumulate = k == s.first ? 0 : 1;
                if (tc::elect_one()) {
                    const uint64_t b = v_desc + st * (kValueBytes >> 4);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int x = 0; x < kSub / 16; ++x)
                            tc::mma_bf16_pair(tmem + j * 128, p_desc + x * 2,
                                              b + j * (kPieceBytes >> 4) + x * (2048 >> 4), kIdescO,
                                              x > 0 ? 1u : accumulate);
                    tc::mma_commit_pair(&v_empty[st], 3);
                    tc::mma_commit_pair(pv_done, 3);
                }
                __syncwarp();
            }
        }
        if (n > 0) tc::mbar_wait_bounded(pv_done, (n - 1) & 1);
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const uint32_t lanes = (uint32_t)warp << 21;  // this warp's quarter of the lanes
        const int row = (warp & 1) * 32 + lane, half = warp >> 1;
        const int row_token = row / p.group, head = head0 + row % p.group;
        auto any_of_both = [&](bool x) {  // of the two warps that share rows
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, "
                "q;\n\t}"
                : "=r"(r)
                : "r"((uint32_t)x), "r"(1 + (warp & 1))
                : "memory");
            return r != 0;
        };
        auto sync_both = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory"); };
        uint32_t n = 0;  // key tiles so far
        while (more(cur)) {
            const Item it = take(p, cur);
            const Subs s = subs_of(it);
            const int tokens = min(max(it.tokens - token0, 0), lp.cta_tokens);  // of this CTA
            const bool valid = row_token < tokens && head < lp.q_heads;
            const int token = it.r.row0 + it.tile * p.tokens_per_tile + token0 + row_token;
            const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile + token0, pos = pos0 + row_token;
            const int hi = p.causal ? min(pos + 1, it.r.kv) : it.r.kv;
            const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
            Branch branch = {0, 0};
            if (kTree && valid) branch = branch_of(p, it.r, token);
            // every row sees keys [lo_all, hi_all): no mask there
            const int hi_all = kTree ? max(it.r.kv - it.r.n, 0) : p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;
            const int lo_all = p.window > 0 ? max(0, pos0 + tokens - p.window) : 0;
            float m = -CUDART_INF_F, l = 0.0f;  // m in powers of two, the same in both threads of a row
            for (int k = s.first; k < s.last; ++k, ++n) {
                const int key0 = k * kSub + half * (kSub / 2);
                wait(&s_full[n & 1], n >> 1 & 1);
                tc::tc_fence_after();
                uint32_t x[32];
                tc::tmem_ld32(tmem + kScores + (n & 1) * (kSub / 2) + lanes, x);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&s_free[n & 1]);
                if (key0 < lo_all || key0 + kSub / 2 > hi_all) {
                    uint32_t seen;
                    if (kTree) {
                        seen = branch.word(key0);
                    } else {
                        const int a = min(max(lo - key0, 0), 32), b = min(max(hi - key0, 0), 32);  // bits a to b - 1
                        seen = (b == 32 ? 0xffffffffu : (1u << b) - 1) & (a == 32 ? 0u : 0xffffffffu << a);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!(seen >> j & 1)) x[j] = 0xff800000u;
                }
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(x[j]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                const bool move = valid && top - m > kLoose;  // also from -inf
                if (any_of_both(k == s.first || move)) {
                    row_max[half * kRows + row] = top;
                    sync_both();
                    const float mn = fmaxf(m, fmaxf(top, row_max[(half ^ 1) * kRows + row]));
                    sync_both();  // (before either is written again)
                    if (k == s.first) {
                        m = mn;
                    } else {
                        const bool up = valid && mn - m > kLoose;
                        const float f = up ? exp2_fast(m - mn) : 1.0f;
                        if (up) m = mn;
                        l *= f;
                        wait(pv_done, (n - 1) & 1);
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 256; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tmem + lanes + c, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st16(tmem + lanes + c, o);
                        }
                        tmem_wait_st();
                    }
                }
                const float base = m == -CUDART_INF_F ? 0.0f : -m;
                const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nb2 = make_float2(base, base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float2 y = make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                    y = fma2(y, sc2, nb2);
                    y.x = exp2_fast(y.x);
                    y.y = exp2_fast(y.y);
                    sum[j & 1] = add2(sum[j & 1], y);
                    x[j] = cvt_bf16x2(y.x, y.y);
                }
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                if (n > 0) wait(pv_done, (n - 1) & 1);  // the probabilities before have been read
                uint8_t* to = ps + row * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4*>(to + (((half * 4 + c) ^ (row & 7)) << 4)) =
                        make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
                tc::fence_proxy_async_smem();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(p_full);
            }
            const bool any = s.first < s.last;
            if (any) {
                wait(pv_done, (n - 1) & 1);
                tc::tc_fence_after();
            }
            row_sum[half * kRows + row] = l;
            sync_both();
            l += row_sum[(half ^ 1) * kRows + row];
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
            const int slot = it.first ? 0 : 1;
            // this thread's 128 columns of each half of 256
            float* part = part_o(p, blockIdx.x, slot) + row * kLatent + half * 128;
            uint16_t* out = p.o + token * p.o_ld + head * p.o_head + half * 128;
#pragma unroll 1
            for (int c = 0; c < 256; c += 16) {
                uint32_t o[16];
                if (any) {
                    tmem_ld16(tmem + lanes + c, o);
                    tc::tmem_wait_ld();
                }
                const int col = (c >> 7) * 256 + (c & 127);
                if (!valid) continue;
                if (it.whole) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = l == 0.0f ? 0u
                                         : cvt_bf16x2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    *reinterpret_cast<uint4*>(out + col) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(out + col + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(part + col + 4 * j) =
                            make_uint4(any ? o[4 * j] : 0, any ? o[4 * j + 1] : 0, any ? o[4 * j + 2] : 0,
                                       any ? o[4 * j + 3] : 0);
                }
            }
            if (half == 0 && row_token < tokens) {
                if (!it.whole)
                    part_ml(p, blockIdx.x, slot)[row] = make_float2(m, l);
                else if (p.lse && valid)
                    p.lse[(int64_t)token * lp.q_heads + head] =
                        l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
            }
            if (!it.whole && threadIdx.x == 0) {
                const Parts parts = parts_of(p, it, start);
                *part_head(p, blockIdx.x, slot) = {parts.last - parts.first + 1, me - parts.first,
                                                   parts.first * 2 + block, 2, tokens * p.group, token, head0};
            }
            tc::tc_fence_before();  // o has been read: the next item's first arrival on p_full says so
            sync_both();            // and the rows' sums may be written again
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync();  // neither CTA's shared or tensor memory is in use by the pair any more
    tc::tc_fence_after();
    if (warp == kMmaWarp) tc::tmem_dealloc_pair(tmem, 512);
}

}  // namespace

cudaError_t launch_latent_pair(const moe_latent_cache& c, const LatentParams& lp, int grid, cudaStream_t st) {
    CUtensorMap qm, km, vm;
    const int k_tokens = c.page_size < kSub / 2 ? c.page_size : kSub / 2, v_tokens = c.page_size < kSub ? c.page_size : kSub;
    if (!make_latent_q_map(&qm, lp) || !make_latent_map(&km, c, c.page_size >= kSub / 2 ? kBlocks : 1, k_tokens) ||
        !make_latent_map(&vm, c, c.page_size >= kSub ? 2 : 1, v_tokens))
        return cudaErrorInvalidValue;
    auto kern = lp.p.tree ? attn_latent_pair_kernel<true> : attn_latent_pair_kernel<false>;
    cudaError_t e = ensure_max_dynamic_smem(kern, kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, kThreads, kSmem, st, lp, qm, km, vm);
}

}  // namespace attn
}  // namespace moe
