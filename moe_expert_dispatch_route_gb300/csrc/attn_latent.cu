// Latent attention, absorbed form: every head's query row of 576 numbers against the same cached rows,
// whose first 512 numbers are the values too.
//
// A query tile has up to 64 rows (tokens x heads of one request) and its keys come 64 at a time:
//   S   = Q K^T      m = 64 rows, n = 64 keys, k = 576      scores, a row per lane
//   O^T += V^T P^T   m = 128 columns (four blocks of them), n = kN rows, k = 64 keys
// The output is transposed, so that 16 to 64 rows fill an instruction's n, and O^T of 64 rows takes 256
// columns of tensor memory (rows as m would take all 512 for 128 rows or as many for 64).  One copy of a key
// row in shared memory serves both products: 128-byte swizzled rows read with k contiguous, and with m
// contiguous.  Two score buffers let the tensor cores work on the next keys' scores while the softmax of
// these runs; probabilities go through shared memory as the second product's B operand.
//
// 65 to 128 heads take two CTAs side by side, each with half of the heads and the same range of
// keys, which the second one to ask finds in L2.
//
// What bounds it: few rows, HBM; 64 rows, the tensor cores: the 36 instructions of a score tile take as
// long with 64 rows as with 128, and the 16 of the product read 6 KB of shared memory each.
//
// The running maximum is followed loosely, as in attn_tile.cuh.
//
//   warps 0-3   softmax (16 rows each), rescaling and epilogue (a lane of tensor memory each)
//   warp 4      issues the MMAs
//   warp 5      copies
#include <cudaTypedefs.h>

#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kLatent = 512, kRope = 64, kWidth = kLatent + kRope;
constexpr int kSub = 64;                       // keys at a time
constexpr int kBlocks = kWidth / 64;           // 128-byte column blocks of a row
constexpr int kBlockBytes = kSub * 128;        // one of them
constexpr int kPieceBytes = 2 * kBlockBytes;   // 128 columns, as the second product takes them
constexpr int kPieces = kLatent / 128;
constexpr int kThreads = 192;

template <int kN>
struct Cfg {
    static constexpr int kQBytes = kBlocks * kN * 128;
    static constexpr int kPBytes = kN * 128;
    // rings of 128-column pieces (four a key tile) and of rotary blocks
    static constexpr int kRing = kN == 64 ? 8 : kN == 32 ? 10 : 11;
    static constexpr int kRopes = kN == 64 ? 2 : 3;
    static constexpr int kBars = 2 * kRing + 2 * kRopes + 2 + 2 + 2 + 2;
    static constexpr int kTail = kBars * 8 + 4 * kRopes + 4 + kN * 20;
    static constexpr int kSmem = 1024 + kQBytes + kPBytes + kRing * kPieceBytes + kRopes * kBlockBytes + kTail;
    static_assert(kSmem <= 232448 - 512, "");
    static_assert(kRing * kPieceBytes >= (kMaxRequests + 32) * 4, "locate()'s scratch");
    // the scores of rows past kN are of what lies behind Q in shared memory, and go nowhere
    static_assert((64 - kN) * 128 <= kPBytes + kRing * kPieceBytes, "");
};

struct LatentParams {
    Params p;      // heads = 1; group = the heads of one CTA
    int q_heads;   // of a token
    int team;      // CTAs that share a range of keys
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

// What the MMA warp has to know of a key tile, put beside it by the copying warp.
enum : uint32_t {
    kNewQ = 1u,    // the first one of a query tile
    kLast = 2u,    // the last one
    kStop = 4u,    // no more
    kSeenLo = 8,   // bits 8-15: first key of the tile that any row sees, 16-23: one past the last
    kSeenHi = 16
};
constexpr uint32_t kIdescAMn = 1u << 15;  // A with its M index contiguous

__device__ __forceinline__ bool any_of_128(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sync_128() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The softmax warps: the sum of n parts of a split tile, those of CTAs first, first + step, ..., in this
// order, a row at a time and four columns a thread.  kEnd: it goes to the output, otherwise to the place of
// the first part.
constexpr int kFan = 4;  // the most parts summed together
template <bool kEnd>
__device__ void join_rows(const LatentParams& lp, const Parts& parts, int first, int step, int n, int block, int rows,
                          const int64_t* row_off, const int64_t* row_lse) {
    const Params& p = lp.p;
    auto cta = [&](int i) { return (first + i * step) * lp.team + block; };
    auto slot = [&](int i) { return part_slot(parts, first + i * step); };
    constexpr int kUnroll = 2;  // rows under way together
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kUnroll) {
        float2 ml[kUnroll][kFan];
        float4 x[kUnroll][kFan];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int i = 0; i < kFan; ++i) {
                ml[u][i] = make_float2(-CUDART_INF_F, 0.0f);
                x[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n && r0 + u < rows) {
                    ml[u][i] = __ldcg(part_ml(p, cta(i), slot(i)) + r0 + u);
                    x[u][i] = __ldcg(reinterpret_cast<const float4*>(part_o(p, cta(i), slot(i)) + (r0 + u) * kLatent) +
                                     threadIdx.x);
                }
            }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u;
            if (r >= rows) break;
            float m = -CUDART_INF_F, l = 0.0f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kFan; ++i) m = fmaxf(m, ml[u][i].x);
            const float to = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
            for (int i = 0; i < kFan; ++i) {
                const float w = exp2_fast(ml[u][i].x - to);
                l += ml[u][i].y * w;
                o.x += x[u][i].x * w, o.y += x[u][i].y * w;
                o.z += x[u][i].z * w, o.w += x[u][i].w * w;
            }
            if (!kEnd) {
                reinterpret_cast<float4*>(part_o(p, cta(0), slot(0)) + r * kLatent)[threadIdx.x] = o;
                continue;
            }
            const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
            if (row_off[r] >= 0)
                *reinterpret_cast<uint2*>(p.o + row_off[r] + threadIdx.x * 4) =
                    make_uint2(cvt_bf16x2(o.x * inv, o.y * inv), cvt_bf16x2(o.z * inv, o.w * inv));
            if (p.lse && row_off[r] >= 0 && threadIdx.x == 0)
                p.lse[row_lse[r]] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
        }
    }
    if (!kEnd) {  // the sums' maxima and sums, once every thread has read the parts'
        sync_128();
        for (int r = threadIdx.x; r < rows; r += 128) {
            float m = -CUDART_INF_F, l = 0.0f;
            for (int i = 0; i < n; ++i) m = fmaxf(m, __ldcg(part_ml(p, cta(i), slot(i)) + r).x);
            const float to = m == -CUDART_INF_F ? 0.0f : m;
            for (int i = 0; i < n; ++i) {
                const float2 ml = __ldcg(part_ml(p, cta(i), slot(i)) + r);
                l += ml.y * exp2_fast(ml.x - to);
            }
            part_ml(p, cta(0), slot(0))[r] = make_float2(m, l);
        }
    }
}

// The softmax warps of a CTA whose part of a split tile is stored: parts are summed kFan at a time, each
// group by the last of its CTAs to arrive, and the sums again (attn_tile.cuh).
template <typename Sync>
__device__ void join(const LatentParams& lp, const Item& it, const Start& st, int me, int block, int rows,
                     const int64_t* row_off, const int64_t* row_lse, int* flag, Sync sync) {
    const Params& p = lp.p;
    const Parts parts = parts_of(p, it, st);
    const int n = parts.last - parts.first + 1, mine = me - parts.first;
    int step = 1;
    for (; step * kFan < n; step *= kFan) {
        const int head = mine / (step * kFan) * (step * kFan), members = min(kFan, (n - head + step - 1) / step);
        if (members == 1) continue;
        const int first = parts.first + head;
        if (!last_of(p.counters + (first + step) * lp.team + block, members, threadIdx.x, flag, sync)) return;
        if (rows > 0) join_rows<false>(lp, parts, first, step, members, block, rows, row_off, row_lse);
    }
    const int members = (n + step - 1) / step;
    if (last_of(p.counters + (parts.first + step) * lp.team + block, members, threadIdx.x, flag, sync) && rows > 0)
        join_rows<true>(lp, parts, parts.first, step, members, block, rows, row_off, row_lse);
}

template <int kN, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
    attn_latent_kernel(const __grid_constant__ LatentParams lp, const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map2) {
    using C = Cfg<kN>;
    const Params& p = lp.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* qs = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);  // by an offset: accesses keep 32-bit addresses
    uint8_t* ps = qs + C::kQBytes;
    uint8_t* ring = ps + C::kPBytes;
    uint8_t* ropes = ring + C::kRing * kPieceBytes;
    int64_t* row_off = reinterpret_cast<int64_t*>(ropes + C::kRopes * kBlockBytes);  // of a row in o, -1: none
    int64_t* row_lse = row_off + kN;
    uint64_t* full = reinterpret_cast<uint64_t*>(row_lse + kN);
    uint64_t* empty = full + C::kRing;
    uint64_t* rope_full = empty + C::kRing;
    uint64_t* rope_empty = rope_full + C::kRopes;
    uint64_t* s_full = rope_empty + C::kRopes;  // [2]
    uint64_t* q_full = s_full + 2;
    uint64_t* q_empty = q_full + 1;
    uint64_t* p_full = q_empty + 1;
    uint64_t* pv_done = p_full + 1;
    uint64_t* done = pv_done + 1;
    uint64_t* never = done + 1;
    float* row_f = reinterpret_cast<float*>(never + 1);  // a row's factor
    uint32_t* cmds = reinterpret_cast<uint32_t*>(row_f + kN);
    __shared__ Start start;
    __shared__ int abort_s, last_s;
    __shared__ uint32_t tmem_s;
    volatile int* abort = &abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int me = blockIdx.x / lp.team, block = blockIdx.x % lp.team;
    constexpr int kMmaWarp = 4, kCopyWarp = 5;
    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int i = 0; i < C::kRing; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kRopes; ++i) {
            tc::mbar_init(&rope_full[i], 1);
            tc::mbar_init(&rope_empty[i], 1);
        }
        tc::mbar_init(&s_full[0], 1);
        tc::mbar_init(&s_full[1], 1);
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_empty, 1);
        tc::mbar_init(p_full, 4);
        tc::mbar_init(pv_done, 1);
        tc::mbar_init(done, 1);
        tc::mbar_init(never, 1);
        tc::fence_barrier_init();
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&map1);
        tc::prefetch_tmap(&map2);
    }
    __syncthreads();
    pdl_begin();
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_s, 512);
        tc::tmem_relinquish();
        tc::tc_fence_before();
    }
    locate<kThreads>(p, reinterpret_cast<uint32_t*>(ring), &start, me, gridDim.x / lp.team);
    tc::tc_fence_after();
    const uint32_t tmem = tmem_s;
    if (p.inject_ns > 0 && blockIdx.x == 0) {  // test hook: the failure path of a bounded wait
        if (threadIdx.x == 0) {
            tc::wait_on_nothing(never, (uint64_t)p.inject_ns);
            set_err(p.err, MOE_ERR_TIMEOUT);
            for (Cursor cur = cursor(start); more(cur);) {  // its parts are counted, as if they had been stored
                const Item it = take(p, cur);
                if (!it.whole) join(lp, it, start, me, block, 0, row_off, row_lse, &last_s, [] {});
            }
        }
        __syncthreads();
        if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
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
    constexpr uint32_t kScores = 4 * kN;  // column of the score buffers, behind O^T

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ copies
        int e = 0, re = 0;
        uint32_t turn = 0, rturn = 0, items = 0, sent = 0, rope_sent = 0, q_sent = 0;
        const int box_keys = min(p.page_size, kSub), npg = kSub / box_keys;
        const bool wide = npg == 1;  // a copy takes both column blocks of a piece
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
            if (items > 0) wait(q_empty, (items - 1) & 1);
            ++items;
            if (!*abort) {
                ++q_sent;
                if (lane == 0) tc::mbar_arrive_expect_tx(q_full, kBlocks * p.tokens_per_tile * p.group * 128);
                __syncwarp();
                if (lane < kBlocks)
                    tc::tma_load_3d(qs + lane * kN * 128, &qmap, q_full, lane * 64, block * p.group,
                                    it.r.row0 + it.tile * p.tokens_per_tile);
            }
            for (int k = s.first; k < s.last; ++k) {
                const int key0 = k * kSub;
                // lane i: page i / (blocks a copy leaves) of the tile
                const int pg = wide ? 0 : lane >> 1;
                const int key = key0 + pg * box_keys, off = key & (p.page_size - 1);
                const bool in = pg < npg && key < it.s.hi && key + box_keys > it.s.lo;
                int page = page_of(p, it, pages, key0, pg);
                if (in && (page < 0 || page >= p.num_pages)) {
                    set_err(p.err, MOE_ERR_BAD_INDEX);
                    page = p.num_pages;  // past the pool: the copy fills zeros
                }
                const bool want = in && (!wide || lane == 0), want1 = in && (wide ? lane == 0 : (lane & 1) == 0);
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, want1)) * (box_keys * 128);
                // the rotary block, and the tile's command
                if (rturn > 0) wait(&rope_empty[re], (rturn - 1) & 1);
                if (lane == 0)
                    cmds[re] = (k == s.first ? kNewQ : 0) | (k == s.last - 1 ? kLast : 0) |
                               (uint32_t)max(it.s.lo - key0, 0) << kSeenLo |
                               (uint32_t)min(it.s.hi - key0, kSub) << kSeenHi;
                if (!*abort) {
                    ++rope_sent;
                    if (lane == 0) tc::mbar_arrive_expect_tx(&rope_full[re], bytes);
                    __syncwarp();
                    if (want1)
                        tc::tma_load_4d(ropes + re * kBlockBytes + pg * box_keys * 128, &map1, &rope_full[re], 0, off,
                                        kLatent / 64, page);
                }
                if (++re == C::kRopes) re = 0, ++rturn;
#pragma unroll 1
                for (int b = 0; b < kPieces; ++b) {
                    if (turn > 0) wait(&empty[e], (turn - 1) & 1);
                    if (!*abort) {
                        ++sent;
                        if (lane == 0) tc::mbar_arrive_expect_tx(&full[e], 2 * bytes);
                        __syncwarp();
                        uint8_t* dst = ring + e * kPieceBytes;
                        if (want) {
                            if (wide)
                                tc::tma_load_4d(dst, &map2, &full[e], 0, off, 2 * b, page);
                            else
                                tc::tma_load_4d(dst + (lane & 1) * kBlockBytes + pg * box_keys * 128, &map1, &full[e],
                                                0, off, 2 * b + (lane & 1), page);
                        }
                    }
                    if (++e == C::kRing) e = 0, ++turn;
                }
                if (k == s.first) ahead();
            }
        }
        if (*abort) {  // copies still in flight land (or a bounded wait gives up) before the CTA ends
            auto landed = [](uint64_t* bars, int n, uint32_t count) {
                for (int i = 0; i < n; ++i) {
                    const uint32_t times = (count + n - 1 - i) / n;  // that entry i has been copied to
                    if (times > 0) tc::mbar_wait_bounded(&bars[i], (times - 1) & 1);
                }
            };
            landed(full, C::kRing, sent);
            landed(rope_full, C::kRopes, rope_sent);
            landed(q_full, 1, q_sent);
        }
        if (rturn > 0) wait(&rope_empty[re], (rturn - 1) & 1);
        if (lane == 0) {
            cmds[re] = kStop;
            tc::mbar_arrive(&rope_full[re]);
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t kIdescS = tc::idesc_bf16_f32(64, kSub);
        constexpr uint32_t kIdescO = tc::idesc_bf16_f32(128, kN) | kIdescAMn;
        int e = 0, re = 0;
        uint32_t turn = 0, rturn = 0, queries = 0, tiles = 0, weighed = 0;
        const uint64_t q_desc = tc::desc_sw128_kmajor(tc::smem_u32(qs));
        const uint64_t p_desc = tc::desc_sw128_kmajor(tc::smem_u32(ps));
        const uint64_t k_desc = tc::desc_sw128_kmajor(tc::smem_u32(ring));
        const uint64_t r_desc = tc::desc_sw128_kmajor(tc::smem_u32(ropes));
        const uint64_t v_desc = desc_sw128_mnmajor(tc::smem_u32(ring), kBlockBytes);
        auto commit = [&](uint64_t* bar) {
            if (tc::elect_one()) tc::mma_commit(bar);
            __syncwarp();
        };
        // the next key tile's command
        auto next = [&]() -> uint32_t {
            wait(&rope_full[re], rturn & 1);
            return cmds[re];
        };
        // its scores, as its pieces arrive; at: its first piece's entry
        auto scores = [&](uint32_t cmd, int& at) {
            if (cmd & kNewQ) wait(q_full, queries++ & 1);
            tc::tc_fence_after();
            const uint32_t to = tmem + kScores + (tiles & 1) * kSub;
            if (tc::elect_one()) {
                const uint64_t a = q_desc + (uint32_t)(8 * (kN * 128 >> 4));
                const uint64_t b = r_desc + (uint32_t)(re * (kBlockBytes >> 4));
#pragma unroll
                for (int s = 0; s < 4; ++s) tc::mma_bf16(to, a + s * 2, b + s * 2, kIdescS, s > 0);
                tc::mma_commit(&rope_empty[re]);
            }
            __syncwarp();
            if (++re == C::kRopes) re = 0, ++rturn;
            const int z0 = cmd >> kSeenLo & 255, z1 = cmd >> kSeenHi & 255;
            at = e;
#pragma unroll 1
            for (int c = 0; c < kPieces; ++c) {
                wait(&full[e], turn & 1);
                if (z0 > 0 || z1 < kSub) {
                    // keys that no row sees hold anything, NaN among it: 0 * NaN would reach o
                    uint4* row = reinterpret_cast<uint4*>(ring + e * kPieceBytes);
                    for (int i = lane; i < kSub * 16; i += 32) {
                        const int r = (i >> 3) & (kSub - 1);
                        if (r < z0 || r >= z1) row[i] = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    const uint64_t a = q_desc + (uint32_t)(2 * c * (kN * 128 >> 4));
                    const uint64_t b = k_desc + (uint32_t)(e * (kPieceBytes >> 4));
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        tc::mma_bf16(to, a + (s / 4) * (kN * 128 >> 4) + (s % 4) * 2,
                                     b + (s / 4) * (kBlockBytes >> 4) + (s % 4) * 2, kIdescS, 1);
                }
                __syncwarp();
                if (++e == C::kRing) e = 0, ++turn;
            }
            commit(&s_full[tiles & 1]);
            if (cmd & kLast) commit(q_empty);
            ++tiles;
        };
        auto values = [&](uint32_t cmd, int at) {
            wait(p_full, weighed++ & 1);
            tc::tc_fence_after();
            const uint32_t accumulate = cmd & kNewQ ? 0 : 1;
            if (tc::elect_one()) {
#pragma unroll 1
                for (int b = 0; b < kPieces; ++b) {
                    const uint64_t a = v_desc + (uint32_t)(at * (kPieceBytes >> 4));
#pragma unroll
                    for (int s = 0; s < kSub / 16; ++s)
                        tc::mma_bf16(tmem + b * kN, a + s * (2048 >> 4), p_desc + s * 2, kIdescO, s > 0 ? 1u : accumulate);
                    tc::mma_commit(&empty[at]);
                    if (++at == C::kRing) at = 0;
                }
                tc::mma_commit(pv_done);
            }
            __syncwarp();
        };
        int at = 0;
        uint32_t cmd = next();
        if (!(cmd & kStop)) scores(cmd, at);
        while (!(cmd & kStop)) {
            // within a query tile the next scores go before this tile's product, which waits for its softmax;
            // those of another query tile wait for its rows, and the product comes first
            const int was = at;
            uint32_t then;
            if (cmd & kLast) {
                values(cmd, was);
                then = next();
                if (!(then & kStop)) scores(then, at);
            } else {
                then = next();
                scores(then, at);
                values(cmd, was);
            }
            cmd = then;
        }
        commit(done);
        tc::mbar_wait_bounded(done, 0);
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const uint32_t lanes = (uint32_t)warp << 21;  // this warp's quarter of the lanes
        const int row = warp * 16 + lane;             // in lanes 0-15
        const bool mine = lane < 16 && row < kN;
        const bool rows_here = warp * 16 < kN;
        uint32_t n = 0;  // key tiles so far
        while (more(cur)) {
            const Item it = take(p, cur);
            const Subs s = subs_of(it);
            const int rows = it.tokens * p.group;
            int lo = 0, hi = 0;
            Branch branch = {0, 0};
            bool valid;
            {
                int64_t off = -1;
                int token = 0, head = 0;
                if (mine && row < rows) {
                    const RowAt at = row_at(p, it, row);
                    token = at.token;
                    head = block * p.group + at.head;
                    if (head < lp.q_heads) off = token * p.o_ld + head * p.o_head;
                }
                valid = off >= 0;
                if (valid) {
                    const int pos = it.r.kv - it.r.n + (token - it.r.row0);
                    hi = p.causal ? min(pos + 1, it.r.kv) : it.r.kv;
                    lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
                    if (kTree) branch = branch_of(p, it.r, token);
                }
                if (mine) {
                    row_off[row] = off;
                    row_lse[row] = (int64_t)token * lp.q_heads + head;
                }
            }
            // every row sees keys [lo_all, hi_all): no mask there
            const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile;
            const int hi_all = kTree ? max(it.r.kv - it.r.n, 0) : p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;
            const int lo_all = p.window > 0 ? max(0, pos0 + it.tokens - p.window) : 0;
            float m = -CUDART_INF_F, l = 0.0f;  // m in powers of two
            for (int k = s.first; k < s.last; ++k, ++n) {
                const int key0 = k * kSub;
                const bool edge = key0 < lo_all || key0 + kSub > hi_all;
                wait(&s_full[n & 1], n >> 1 & 1);
                tc::tc_fence_after();
                uint32_t x[kSub];
                float mn = m;
                if (rows_here) {
                    const uint32_t ts = tmem + kScores + (n & 1) * kSub + lanes;
                    tc::tmem_ld32(ts, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
                    tc::tmem_ld32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
                    tc::tmem_wait_ld();
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < kSub; ++j) {
                            const int key = key0 + j;
                            if (key < lo || key >= hi || (kTree && !branch.sees(key))) x[j] = 0xff800000u;
                        }
                    }
                    float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int j = 0; j < kSub; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(x[j]));
                    mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2);
                }
                const bool move = valid && mn - m > kLoose;  // also from -inf
                if (k == s.first) {
                    m = mn;
                } else if (any_of_128(move)) {
                    const float f = move ? exp2_fast(m - mn) : 1.0f;
                    if (move) m = mn;
                    l *= f;
                    if (mine) row_f[row] = f;
                    sync_128();
                    wait(pv_done, (n - 1) & 1);
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4 * kN; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(tmem + lanes + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * row_f[(c + j) % kN]);
                        tmem_st16(tmem + lanes + c, o);
                    }
                    tmem_wait_st();
                }
                if (rows_here) {
                    const float base = m == -CUDART_INF_F ? 0.0f : m;
                    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nb2 = make_float2(-base, -base);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int j = 0; j < kSub / 2; ++j) {
                        float2 y = make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                        y = fma2(y, sc2, nb2);
                        y.x = exp2_fast(y.x);
                        y.y = exp2_fast(y.y);
                        sum[j & 1] = add2(sum[j & 1], y);
                        x[j] = cvt_bf16x2(y.x, y.y);
                    }
                    sum[0] = add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                }
                if (n > 0) wait(pv_done, (n - 1) & 1);  // the probabilities before have been read
                if (mine) {
                    uint8_t* to = ps + row * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4*>(to + ((c ^ (row & 7)) << 4)) =
                            make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
                    tc::fence_proxy_async_smem();
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(p_full);
            }
            const bool any = s.first < s.last;
            if (any) {
                wait(pv_done, (n - 1) & 1);
                tc::tc_fence_after();
            }
            const int slot = it.first ? 0 : 1;
            if (mine) {
                if (it.whole) {
                    row_f[row] = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                    if (p.lse && row_off[row] >= 0)
                        p.lse[row_lse[row]] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
                } else if (row < rows) {
                    part_ml(p, blockIdx.x, slot)[row] = make_float2(m, l);
                }
            }
            sync_128();  // the rows' factors and places
            // this thread's column of each block of 128, 16 rows at a time
            float* part = part_o(p, blockIdx.x, slot) + warp * 32 + lane;
#pragma unroll 1
            for (int b = 0; b < kPieces; ++b)
#pragma unroll 1
                for (int r0 = 0; r0 < rows; r0 += 16) {
                    uint32_t o[16];
                    if (any) {
                        tmem_ld16(tmem + lanes + b * kN + r0, o);
                        tc::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = 0;
                    }
                    if (!it.whole) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (r0 + j < rows) part[(r0 + j) * kLatent + b * 128] = __uint_as_float(o[j]);
                        continue;
                    }
                    // neighbours trade values: an even lane stores two columns of one row, an odd one of the next
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float f0 = row_f[r0 + j], f1 = row_f[r0 + j + 1];
                        const float v0 = f0 == 0.0f ? 0.0f : __uint_as_float(o[j]) * f0;
                        const float v1 = f1 == 0.0f ? 0.0f : __uint_as_float(o[j + 1]) * f1;
                        const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? v0 : v1, 1);
                        const int64_t off = row_off[r0 + j + (lane & 1)];
                        if (off >= 0)
                            *reinterpret_cast<uint32_t*>(p.o + off + b * 128 + warp * 32 + (lane & 30)) =
                                lane & 1 ? cvt_bf16x2(got, v1) : cvt_bf16x2(v0, got);
                    }
                }
            if (!it.whole) join(lp, it, start, me, block, rows, row_off, row_lse, &last_s, sync_128);
            tc::tc_fence_before();  // o has been read: the next item's first arrival on p_full says so
            sync_128();             // and the rows' places may be written again
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// q as (d, head, token): a box holds the rows of a query tile in (token, head) order.
bool make_q_map(CUtensorMap* m, const Params& p, int q_heads) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    cuuint64_t dims[3] = {kWidth, (cuuint64_t)q_heads, (cuuint64_t)p.T};
    cuuint64_t strides[2] = {(cuuint64_t)(q_heads > 1 ? p.q_head * 2 : kWidth * 2),
                             (cuuint64_t)(p.T > 1 ? p.q_ld * 2 : kWidth * 2)};
    cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)p.tokens_per_tile};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The pool as (d within a block, token, column block, page): a box holds `blocks` column blocks of up to
// kSub tokens.
bool make_latent_map(CUtensorMap* m, const moe_latent_cache& c, int blocks) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    cuuint64_t dims[4] = {64, (cuuint64_t)c.page_size, kBlocks, (cuuint64_t)c.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)c.stride_token * 2, 128, (cuuint64_t)c.stride_page * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < kSub ? c.page_size : kSub), (cuuint32_t)blocks, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, c.kv, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int kN, bool kTree>
cudaError_t launch_as(const moe_latent_cache& c, const LatentParams& lp, int grid, cudaStream_t st) {
    CUtensorMap qm, m1, m2;
    if (!make_q_map(&qm, lp.p, lp.q_heads) || !make_latent_map(&m1, c, 1) || !make_latent_map(&m2, c, 2))
        return cudaErrorInvalidValue;
    auto kern = attn_latent_kernel<kN, kTree>;
    cudaError_t e = ensure_max_dynamic_smem(kern, Cfg<kN>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, kThreads, Cfg<kN>::kSmem, st, lp, qm, m1, m2);
}
template <bool kTree>
cudaError_t launch_of(const moe_latent_cache& c, const LatentParams& lp, int rows, int grid, cudaStream_t st) {
    return rows <= 16   ? launch_as<16, kTree>(c, lp, grid, st)
           : rows <= 32 ? launch_as<32, kTree>(c, lp, grid, st)
                        : launch_as<64, kTree>(c, lp, grid, st);
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_latent(const moe_latent_cache& c, const moe_attn_args& a, const uint64_t* tree, int grid_cap,
                               cudaStream_t st) {
    using namespace attn;
    LatentParams lp;
    Params& p = lp.p;
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
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.page_shift = 0;
    while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.causal = tree ? 0 : a.causal;
    p.window = a.window < kMaxTokens ? a.window : kMaxTokens;
    p.tree = tree;
    p.err = a.err_flag;
    p.counters = static_cast<uint32_t*>(a.workspace);
    p.parts = static_cast<uint8_t*>(a.workspace) + kMaxCtas * sizeof(uint32_t);
    p.inject_ns = wait_injection_ns();
    lp.q_heads = a.num_q_heads;
    lp.team = a.num_q_heads > 64 ? 2 : 1;
    p.heads = 1;
    p.group = (a.num_q_heads + lp.team - 1) / lp.team;
    // a request's rows in as few tiles as hold them, of 64 at most; a narrow tile where they are few
    const int most = 64 / p.group;
    p.tokens_per_tile = a.max_q < most ? a.max_q : most;
    p.item_cost = 2;
    p.item_slack = 1;
    p.cta_units = 2;
    if (grid_cap > kMaxCtas) grid_cap = kMaxCtas;
    const int teams = grid_cap / lp.team < 1 ? 1 : grid_cap / lp.team;
    int grid = grid_for(p, teams);
    const int fit = device_info().num_sms / lp.team;
    if (grid > fit) grid = fit;
    const int rows = p.tokens_per_tile * p.group;
    return tree ? launch_of<true>(c, lp, rows, grid * lp.team, st) : launch_of<false>(c, lp, rows, grid * lp.team, st);
}

}  // namespace moe
