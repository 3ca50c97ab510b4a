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
// Requests of more rows go to attn_latent_pair.cu.
//
// What bounds it: HBM where rows are few (64 requests of up to 16384 tokens, 16 heads: 101-105 us, 5.7 TB/s; 32 heads
// 109), and shared memory next to it: for 64 keys the scores' 36 instructions read 144 KB of operands, the product's 16
// 64 KB and the probabilities, transposed operands at half the rate, and the copies write 72 KB, 2750 cycles for 16
// rows and 3000 for 64 at 128 bytes a cycle, where HBM takes 3130.  One request of 1501 tokens, 16 heads: 16.8 us, a
// chain of loads, one or two key tiles, and the second kernel (4 us).
//
// The running maximum is followed loosely, as in attn_tile.cuh.
//
//   warps 0-3   softmax (16 rows each), rescaling and epilogue (a lane of tensor memory each)
//   warp 4      issues the scores' MMAs
//   warp 5      issues the products' MMAs: from one warp, each product would wait for the copies of the scores
//               behind it, which wait for the product to give their place back
//   warps 6, 7  copies: the rotary blocks and half of the pieces, the other half (a copying warp issues
//               a copy about every 100 cycles, and 16-token pages take 36 of them for 64 keys)
#include "attn_latent.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;

template <int kN>
struct Cfg {
    static constexpr int kQBytes = kBlocks * kN * 128;
    static constexpr int kPBytes = kN * 128;
    // rings of 128-column pieces (four a key tile) and of rotary blocks
    static constexpr int kRing = kN == 64 ? 8 : 10;
    static constexpr int kRopes = kN == 64 ? 2 : 3;
    static constexpr int kBars = 2 * kRing + 2 * kRopes + 4 + 2 + 2 + 2;
    static constexpr int kTail = kBars * 8 + 4 * kRopes + 4 + kN * 20;
    static constexpr int kSmem = 1024 + kQBytes + kPBytes + kRing * kPieceBytes + kRopes * kBlockBytes + kTail;
    static_assert(kSmem <= 232448 - 512, "");
    static_assert(kRing % 2 == 0, "the copying warps' halves of a tile");
    static_assert(kRing * kPieceBytes >= (kMaxRequests + 32) * 4, "locate()'s scratch");
    // the scores of rows past kN are of what lies behind Q in shared memory, and go nowhere
    static_assert((64 - kN) * 128 <= kPBytes + kRing * kPieceBytes, "");
};

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
// 16 lanes, 64 columns from taddr: of lane g = lane / 4 (r[4 i], r[4 i + 1]) and of lane g + 8 (r[4 i + 2], r[4 i + 3])
// the columns 8 i + 2 (lane % 4) and the next.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ float max_of_4(float v) {  // of the lanes that share a row
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ void sync_128() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Split tiles, put together: the CTAs of a slot each take a share of their tile's output, so that a long context's
// many parts are read by as many CTAs.  (Joined by the last CTA to arrive, as in attn_tile.cuh, a tile of 64 rows took
// its CTA 15 to 30 us, 128 KB a part from a busy memory, and one request of 100000 tokens with 128 heads 97 us, 54
// so.)  This kernel takes 4 us for one request and 8 to 15 where every CTA has a part; where no tile can be split it is
// left out (one request of 200 tokens 15.6 -> 14.4 us).
// A thread takes four columns of a row; a small share with many parts is shared by several groups of
// threads, whose sums are added in order.
constexpr int kJoinThreads = 512;
constexpr int kMostParts = 160;  // of a tile, and CTAs of a call
__device__ __forceinline__ void join_share(const LatentParams& lp, const PartHead& h, float* weights, float4* sums) {
    const Params& p = lp.p;
    const int tid = threadIdx.x;
    constexpr int kPer = kLatent / 4;
    const int total = h.rows * kPer, e0 = (int)((int64_t)total * h.rank / h.n);
    const int count = (int)((int64_t)total * (h.rank + 1) / h.n) - e0;
    if (count == 0) return;
    const uint8_t* base = p.parts + ((size_t)h.first * 2 + 1) * kPartBytes;
    const size_t stride = (size_t)h.step * 2 * kPartBytes;
    auto part_at = [&](int i) { return base + i * stride - (i == 0 ? kPartBytes : 0); };
    auto ml_at = [&](int i, int r) {
        return __ldcg(reinterpret_cast<const float2*>(part_at(i) + (size_t)kMaxRows * 128 * 4) + r);
    };
    const int r0 = e0 / kPer, nrows = (e0 + count - 1) / kPer - r0 + 1;
    auto load = [&](int i, int e) { return __ldcg(reinterpret_cast<const float4*>(part_at(i)) + e); };
    const bool wide = count > kJoinThreads;  // several numbers a thread, of few parts
    int groups = 1;
    while (groups * 2 * count <= kJoinThreads && groups * 4 <= h.n) groups *= 2;
    // the first numbers are on their way while the weights are found: a chain of two loads in all
    constexpr int kE = 4, kI = 2, kP = 8;  // elements and parts under way together, and parts of one element
    float4 x[kE][kI];
    auto fetch = [&](int at, int i0) {
#pragma unroll
        for (int u = 0; u < kE; ++u)
#pragma unroll
            for (int i = 0; i < kI; ++i)
                if (at + u * kJoinThreads < count && i0 + i < h.n) x[u][i] = load(i0 + i, e0 + at + u * kJoinThreads);
    };
    if (wide) fetch(tid, 0);
    // a warp a row, a lane a part (or several): its weight
    constexpr int kPerLane = kMostParts / 32, kPerWarp = 64 / (kJoinThreads / 32);
    const int lane = tid & 31;
    auto weigh = [&](int row, const float2 (&ml)[kPerLane], int parts) {
        float m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) m = i < parts ? fmaxf(m, ml[i].x) : m;
        m = warp_max(m);
        const float to = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) l += i < parts ? ml[i].y * exp2_fast(ml[i].x - to) : 0.0f;
        l = warp_sum(l);
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (i < parts) weights[(row - r0) * h.n + i * 32 + lane] = exp2_fast(ml[i].x - to) * inv;
        const int token = h.token + row / p.group, head = h.head + row % p.group;
        if (lane == 0 && p.lse && head < lp.q_heads && row * kPer >= e0 && row * kPer < e0 + count)
            p.lse[(int64_t)token * lp.q_heads + head] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
    };
    const int parts = h.n > lane ? (h.n - lane + 31) / 32 : 0;  // of this lane
    if (h.n <= 32) {
        float2 ml[kPerWarp];
#pragma unroll
        for (int k = 0; k < kPerWarp; ++k) {
            const int r = (tid >> 5) + k * (kJoinThreads / 32);
            if (r < nrows && parts > 0) ml[k] = ml_at(lane, r0 + r);
        }
#pragma unroll
        for (int k = 0; k < kPerWarp; ++k) {
            const int r = (tid >> 5) + k * (kJoinThreads / 32);
            if (r < nrows) {
                const float2 one[kPerLane] = {ml[k]};
                weigh(r0 + r, one, min(parts, 1));
            }
        }
    } else if (tid >> 5 < nrows) {  // a share of at most 3 rows
        float2 ml[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
            if (i < parts) ml[i] = ml_at(i * 32 + lane, r0 + (tid >> 5));
        weigh(r0 + (tid >> 5), ml, parts);
    }
    __syncthreads();
    auto out = [&](int e, float4 o) {
        const int row = e / kPer, token = h.token + row / p.group, head = h.head + row % p.group;
        if (head < lp.q_heads)
            *reinterpret_cast<uint2*>(p.o + token * p.o_ld + head * p.o_head + e % kPer * 4) =
                make_uint2(cvt_bf16x2(o.x, o.y), cvt_bf16x2(o.z, o.w));
    };
    auto add = [](float4& o, float4 x, float w) {
        if (w == 0.0f) return;  // a part without keys for this row: its numbers may be anything
        o.x += x.x * w, o.y += x.y * w, o.z += x.z * w, o.w += x.w * w;
    };
    if (wide) {
        for (int at = tid; at < count; at += kE * kJoinThreads) {
            float4 o[kE];
#pragma unroll
            for (int u = 0; u < kE; ++u) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < h.n; i0 += kI) {
                if (at >= kE * kJoinThreads || i0 > 0) fetch(at, i0);
#pragma unroll
                for (int u = 0; u < kE; ++u)
#pragma unroll
                    for (int i = 0; i < kI; ++i)
                        if (at + u * kJoinThreads < count && i0 + i < h.n)
                            add(o[u], x[u][i], weights[((e0 + at + u * kJoinThreads) / kPer - r0) * h.n + i0 + i]);
            }
#pragma unroll
            for (int u = 0; u < kE; ++u)
                if (at + u * kJoinThreads < count) out(e0 + at + u * kJoinThreads, o[u]);
        }
        return;
    }
    const int per = kJoinThreads / groups, g = tid / per, at = tid % per;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at < count) {
        const float* w = weights + ((e0 + at) / kPer - r0) * h.n;
        for (int i0 = g; i0 < h.n; i0 += kP * groups) {
            float4 y[kP];
#pragma unroll
            for (int i = 0; i < kP; ++i)
                if (i0 + i * groups < h.n) y[i] = load(i0 + i * groups, e0 + at);
#pragma unroll
            for (int i = 0; i < kP; ++i)
                if (i0 + i * groups < h.n) add(o, y[i], w[i0 + i * groups]);
        }
    }
    sums[tid] = o;
    __syncthreads();
    if (g == 0 && at < count) {
        for (int i = 1; i < groups; ++i) add(o, sums[i * per + at], 1.0f);
        out(e0 + at, o);
    }
}

// ctas: of the first kernel.
__global__ void __launch_bounds__(kJoinThreads) attn_latent_join_kernel(const __grid_constant__ LatentParams lp, int ctas) {
    __shared__ float weights[64 + 2 * kMostParts];  // [row of the share][part]
    __shared__ float4 sums[kJoinThreads];
    pdl_begin();
    for (int i = blockIdx.x; i < 2 * ctas; i += gridDim.x) {
        const PartHead h = *part_head(lp.p, i >> 1, i & 1);
        if (h.n > 0) join_share(lp, h, weights, sums);
        __syncthreads();
    }
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
    uint64_t* s_free = s_full + 2;              // [2]
    uint64_t* q_full = s_free + 2;
    uint64_t* q_empty = q_full + 1;
    uint64_t* p_full = q_empty + 1;
    uint64_t* pv_done = p_full + 1;
    uint64_t* done = pv_done + 1;
    uint64_t* never = done + 1;
    float* row_f = reinterpret_cast<float*>(never + 1);  // a row's factor
    uint32_t* cmds = reinterpret_cast<uint32_t*>(row_f + kN);
    __shared__ Start start;
    __shared__ int abort_s;
    __shared__ uint32_t tmem_s;
    volatile int* abort = &abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMmaWarp = 4, kValueWarp = 5, kCopyWarp = 6;
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
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s_full[i], 1);
            tc::mbar_init(&s_free[i], 4);
        }
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
    locate<kThreads>(p, reinterpret_cast<uint32_t*>(ring), &start);
    tc::tc_fence_after();
    const uint32_t tmem = tmem_s;
    if (threadIdx.x < 2) part_head(p, blockIdx.x, threadIdx.x)->n = 0;
    __syncthreads();
    if (p.inject_ns > 0 && blockIdx.x == 0) {  // test hook: the failure path of a bounded wait
        if (threadIdx.x == 0) {
            tc::wait_on_nothing(never, (uint64_t)p.inject_ns);
            set_err(p.err, MOE_ERR_TIMEOUT);
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

    if (warp >= kCopyWarp) {
        // ------------------------------------------------------------ copies
        const bool first_warp = warp == kCopyWarp;  // takes Q, the rotary blocks and pieces 0 and 1
        int e = first_warp ? 0 : 2, re = 0;
        uint32_t tiles = 0, items = 0, q_sent = 0, rope_sent = 0, sent = 0;  // sent: pairs of pieces
        const int box_keys = min(p.page_size, kSub), npg = kSub / box_keys;
        const bool wide = npg == 1;  // a copy takes both column blocks of a piece
        // keys are read once here: they leave L2 to the parts of split tiles (16 heads: 104 us, 108 without)
        const uint64_t policy = tc::policy_of(true);
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
            if (first_warp) {
                if (items > 0) wait(q_empty, (items - 1) & 1);
                ++items;
                if (!*abort) {
                    ++q_sent;
                    if (lane == 0) tc::mbar_arrive_expect_tx(q_full, kBlocks * p.tokens_per_tile * p.group * 128);
                    __syncwarp();
                    if (lane < kBlocks)
                        tc::tma_load_3d(qs + lane * kN * 128, &qmap, q_full, lane * 64, 0,
                                        it.r.row0 + it.tile * p.tokens_per_tile);
                }
            }
            for (int k = s.first; k < s.last; ++k, ++tiles) {
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
                if (first_warp) {
                    // the rotary block, and the tile's command
                    const uint32_t turn = tiles / C::kRopes;
                    if (turn > 0) wait(&rope_empty[re], (turn - 1) & 1);
                    if (lane == 0)
                        cmds[re] = (k == s.first ? kNewQ : 0) | (k == s.last - 1 ? kLast : 0) |
                                   (uint32_t)max(it.s.lo - key0, 0) << kSeenLo |
                                   (uint32_t)min(it.s.hi - key0, kSub) << kSeenHi;
                    if (!*abort) {
                        ++rope_sent;
                        if (lane == 0) tc::mbar_arrive_expect_tx(&rope_full[re], bytes);
                        __syncwarp();
                        if (want1)
                            tc::tma_load_4d_hint(ropes + re * kBlockBytes + pg * box_keys * 128, &map1, &rope_full[re],
                                                 0, off, kLatent / 64, page, policy);
                    }
                    if (++re == C::kRopes) re = 0;
                }
#pragma unroll 1
                for (int b = first_warp ? 0 : 2, end = b + 2; b < end; ++b) {
                    const uint32_t turn = (tiles * kPieces + b) / C::kRing;
                    if (turn > 0) wait(&empty[e], (turn - 1) & 1);
                    if (!*abort) {
                        sent = tiles + 1;
                        if (lane == 0) tc::mbar_arrive_expect_tx(&full[e], 2 * bytes);
                        __syncwarp();
                        uint8_t* dst = ring + e * kPieceBytes;
                        if (want) {
                            if (wide)
                                tc::tma_load_4d_hint(dst, &map2, &full[e], 0, off, 2 * b, page, policy);
                            else
                                tc::tma_load_4d_hint(dst + (lane & 1) * kBlockBytes + pg * box_keys * 128, &map1,
                                                     &full[e], 0, off, 2 * b + (lane & 1), page, policy);
                        }
                    }
                    if (++e >= C::kRing) e -= C::kRing;
                }
                e = e + 2 < C::kRing ? e + 2 : e + 2 - C::kRing;  // the other warp's
                if (k == s.first) ahead();
            }
        }
        if (*abort) {  // copies still in flight land (or a bounded wait gives up) before the CTA ends
            for (int i = 0; i < C::kRopes; ++i) {
                const uint32_t times = (rope_sent + C::kRopes - 1 - i) / C::kRopes;  // that entry i has been copied to
                if (times > 0) tc::mbar_wait_bounded(&rope_full[i], (times - 1) & 1);
            }
            if (q_sent > 0) tc::mbar_wait_bounded(q_full, (q_sent - 1) & 1);
            // this warp's pieces of the last tiles; those before lie in the same entries
            for (uint32_t t = sent, i = 0; t-- > 0 && i < C::kRing / 2; ++i)
                for (int b = first_warp ? 0 : 2, end = b + 2; b < end; ++b) {
                    const uint32_t x = t * kPieces + b;
                    tc::mbar_wait_bounded(&full[x % C::kRing], x / C::kRing & 1);
                }
        }
        if (first_warp) {
            const uint32_t turn = tiles / C::kRopes;
            if (turn > 0) wait(&rope_empty[re], (turn - 1) & 1);
            if (lane == 0) {
                cmds[re] = kStop;
                tc::mbar_arrive(&rope_full[re]);
            }
        }    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ the scores' MMAs
        constexpr uint32_t kIdescS = tc::idesc_bf16_f32(64, kSub);
        int e = 0, re = 0;
        uint32_t turn = 0, rturn = 0, queries = 0, tiles = 0;
        const uint64_t q_desc = tc::desc_sw128_kmajor(tc::smem_u32(qs));
        const uint64_t k_desc = tc::desc_sw128_kmajor(tc::smem_u32(ring));
        const uint64_t r_desc = tc::desc_sw128_kmajor(tc::smem_u32(ropes));
        auto commit = [&](uint64_t* bar) {
            if (tc::elect_one()) tc::mma_commit(bar);
            __syncwarp();
        };
        // the next key tile's command
        auto next = [&]() -> uint32_t {
            wait(&rope_full[re], rturn & 1);
            return cmds[re];
        };
        // its scores, as its pieces arrive
        auto scores = [&](uint32_t cmd) {
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
        for (;;) {
            const uint32_t cmd = next();
            if (cmd & kStop) break;
            if (tiles > 1) wait(&s_free[tiles & 1], (tiles >> 1) - 1 & 1);  // the buffer's scores before have been read
            scores(cmd);
        }
        commit(done);
        tc::mbar_wait_bounded(done, 0);
    } else if (warp == kValueWarp) {
        // ------------------------------------------------------------ the products' MMAs
        constexpr uint32_t kIdescO = tc::idesc_bf16_f32(128, kN) | kIdescAMn;
        const uint64_t p_desc = tc::desc_sw128_kmajor(tc::smem_u32(ps));
        const uint64_t v_desc = desc_sw128_mnmajor(tc::smem_u32(ring), kBlockBytes);
        int at = 0;
        uint32_t n = 0;  // key tiles so far
        while (more(cur)) {
            const Item it = take(p, cur);
            const Subs s = subs_of(it);
            for (int k = s.first; k < s.last; ++k, ++n) {
                wait(p_full, n & 1);
                tc::tc_fence_after();
                const uint32_t accumulate = k == s.first ? 0 : 1;
                if (tc::elect_one()) {
#pragma unroll
                    for (int b = 0; b < kPieces; ++b) {
                        const int e = at + b < C::kRing ? at + b : at + b - C::kRing;
                        const uint64_t a = v_desc + (uint32_t)(e * (kPieceBytes >> 4));
#pragma unroll
                        for (int x = 0; x < kSub / 16; ++x)
                            tc::mma_bf16(tmem + b * kN, a + x * (2048 >> 4), p_desc + x * 2, kIdescO,
                                         x > 0 ? 1u : accumulate);
                        tc::mma_commit(&empty[e]);
                    }
                    tc::mma_commit(pv_done);
                }
                __syncwarp();
                at = at + kPieces < C::kRing ? at + kPieces : at + kPieces - C::kRing;
            }
        }
        if (n > 0) tc::mbar_wait_bounded(pv_done, (n - 1) & 1);
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        const uint32_t lanes = (uint32_t)warp << 21;  // this warp's quarter of the lanes
        // scores: rows g and g + 8 of the warp's 16, a quarter of the columns of each
        const int row0 = warp * 16 + (lane >> 2);
        const bool rows_here = warp * 16 < kN, speaks = rows_here && (lane & 3) == 0;
        uint32_t n = 0;  // key tiles so far
        while (more(cur)) {
            const Item it = take(p, cur);
            const Subs s = subs_of(it);
            const int rows = it.tokens * p.group;
            int lo[2] = {0, 0}, hi[2] = {0, 0};
            Branch branch[2] = {{0, 0}, {0, 0}};
            bool valid[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = row0 + 8 * i;
                const RowAt at = row_at(p, it, min(row, rows - 1));
                valid[i] = row < rows;
                if (valid[i]) {
                    const int pos = it.r.kv - it.r.n + (at.token - it.r.row0);
                    hi[i] = p.causal ? min(pos + 1, it.r.kv) : it.r.kv;
                    lo[i] = p.window > 0 ? max(0, pos - p.window + 1) : 0;
                    if (kTree) branch[i] = branch_of(p, it.r, at.token);
                }
                if (speaks) {
                    row_off[row] = valid[i] ? at.token * p.o_ld + at.head * p.o_head : -1;
                    row_lse[row] = (int64_t)at.token * lp.q_heads + at.head;
                }
            }
            // every row sees keys [lo_all, hi_all): no mask there
            const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile;
            const int hi_all = kTree ? max(it.r.kv - it.r.n, 0) : p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;
            const int lo_all = p.window > 0 ? max(0, pos0 + it.tokens - p.window) : 0;
            // m in powers of two, the same in the four lanes of a row; l of this lane's columns
            float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.0f, 0.0f};
            for (int k = s.first; k < s.last; ++k, ++n) {
                const int key0 = k * kSub;
                wait(&s_full[n & 1], n >> 1 & 1);
                tc::tc_fence_after();
                uint32_t x[32];
                float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
                if (rows_here) {
                    tmem_ld_16x64(tmem + kScores + (n & 1) * kSub + lanes, x);
                    tc::tmem_wait_ld();
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&s_free[n & 1]);
                if (rows_here) {
                    if (key0 < lo_all || key0 + kSub > hi_all) {
                        const int col = (lane & 3) * 2;
                        uint32_t seen[2][2];  // of a row, from this lane's first column on: 32 keys, and the next 32
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                seen[i][u] = kTree && valid[i] ? branch[i].word(key0 + u * 32 + col) : 0u;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int at = (j >> 2) * 8 + (j & 1), key = key0 + col + at, i = j >> 1 & 1;
                            if (kTree ? !(seen[i][at >> 5] >> (at & 31) & 1) : key < lo[i] || key >= hi[i])
                                x[j] = 0xff800000u;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) mx[j >> 1 & 1] = fmaxf(mx[j >> 1 & 1], __uint_as_float(x[j]));
                }
                bool move = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[i] *= p.scale_log2;
                    move |= valid[i] && mx[i] - m[i] > kLoose;  // also from -inf
                }
                if (k == s.first) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) m[i] = max_of_4(mx[i]);
                } else if (any_of_128(move)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mn = max_of_4(mx[i]);
                        const bool up = valid[i] && mn - m[i] > kLoose;
                        const float f = up ? exp2_fast(m[i] - mn) : 1.0f;
                        if (up) m[i] = mn;
                        l[i] *= f;
                        if (speaks) row_f[row0 + 8 * i] = f;
                    }
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
                    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
                    float2 nb2[2], sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float base = m[i] == -CUDART_INF_F ? 0.0f : -m[i];
                        nb2[i] = make_float2(base, base);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float2 y = make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                        y = fma2(y, sc2, nb2[j & 1]);
                        y.x = exp2_fast(y.x);
                        y.y = exp2_fast(y.y);
                        sum[j & 1] = add2(sum[j & 1], y);
                        x[j] = cvt_bf16x2(y.x, y.y);
                    }
                    l[0] += sum[0].x + sum[0].y;
                    l[1] += sum[1].x + sum[1].y;
                }
                if (n > 0) wait(pv_done, (n - 1) & 1);  // the probabilities before have been read
                if (rows_here) {
                    uint8_t* to = ps + row0 * 128 + (lane & 3) * 4;  // (row0 + 8) & 7 is row0 & 7
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int at = (c ^ (row0 & 7)) << 4;
                        *reinterpret_cast<uint32_t*>(to + at) = x[2 * c];
                        *reinterpret_cast<uint32_t*>(to + 1024 + at) = x[2 * c + 1];
                    }
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
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                const int row = row0 + 8 * i;
                if (!speaks) continue;
                if (it.whole) {
                    row_f[row] = l[i] > 0.0f ? 1.0f / l[i] : (l[i] == 0.0f ? 0.0f : l[i]);
                    if (p.lse && valid[i])
                        p.lse[row_lse[row]] = l[i] == 0.0f ? -CUDART_INF_F : (m[i] + log2f(l[i])) * 0.6931471805599453f;
                } else if (row < rows) {
                    part_ml(p, blockIdx.x, slot)[row] = make_float2(m[i], l[i]);
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
            if (!it.whole && threadIdx.x == 0) {
                const Parts parts = parts_of(p, it, start);
                *part_head(p, blockIdx.x, slot) = {parts.last - parts.first + 1, (int)blockIdx.x - parts.first, parts.first, 1,
                                                   rows, it.r.row0 + it.tile * p.tokens_per_tile, 0};
            }
            tc::tc_fence_before();  // o has been read: the next item's first arrival on p_full says so
            sync_128();             // and the rows' places may be written again
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

template <int kN, bool kTree>
cudaError_t launch_as(const moe_latent_cache& c, const LatentParams& lp, int grid, cudaStream_t st) {
    CUtensorMap qm, m1, m2;
    const int tokens = c.page_size < kSub ? c.page_size : kSub;
    if (!make_latent_q_map(&qm, lp) || !make_latent_map(&m1, c, 1, tokens) || !make_latent_map(&m2, c, 2, tokens))
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

bool make_latent_q_map(CUtensorMap* m, const LatentParams& lp) {
    const Params& p = lp.p;
    const int q_heads = lp.q_heads;
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    cuuint64_t dims[3] = {kWidth, (cuuint64_t)q_heads, (cuuint64_t)p.T};
    cuuint64_t strides[2] = {(cuuint64_t)(q_heads > 1 ? p.q_head * 2 : kWidth * 2),
                             (cuuint64_t)(p.T > 1 ? p.q_ld * 2 : kWidth * 2)};
    cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)lp.cta_tokens};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_latent_map(CUtensorMap* m, const moe_latent_cache& c, int blocks, int tokens) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    cuuint64_t dims[4] = {64, (cuuint64_t)c.page_size, kBlocks, (cuuint64_t)c.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)c.stride_token * 2, 128, (cuuint64_t)c.stride_page * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)tokens, (cuuint32_t)blocks, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, c.kv, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

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
    p.heads = 1;
    // Up to 64 rows a request go to one CTA, more to pairs, which take two thirds of the time for 128 rows that
    // single CTAs take for 64 twice (128 heads: 150 us against 201).  One rule for the whole call, as in attn.cu.
    const bool pairs = (int64_t)a.max_q * a.num_q_heads > 64;
    lp.split_heads = a.num_q_heads > 64;
    p.group = lp.split_heads ? (a.num_q_heads + 1) / 2 : a.num_q_heads;
    const int most = 64 / p.group, half = a.max_q / 2 + a.max_q % 2;  // tokens
    lp.cta_tokens = !pairs ? a.max_q : lp.split_heads ? 1 : half < most ? half : most;
    p.tokens_per_tile = pairs && !lp.split_heads ? 2 * lp.cta_tokens : lp.cta_tokens;
    // what a query tile costs beside its key tiles (1.7 us each 64 keys) is about 4 us
    p.item_cost = 1;
    p.item_slack = 1;
    p.cta_units = 1;
    const int max_ctas = grid_cap;
    if (grid_cap > kMostParts) grid_cap = kMostParts;
    int grid = device_info().num_sms < grid_cap ? device_info().num_sms : grid_cap;
    const int team = pairs ? 2 : 1, teams = grid / team > 0 ? grid / team : 1;
    grid = grid_for(p, teams) * team;
    const int rows = p.tokens_per_tile * p.group;
    const cudaError_t e = pairs  ? launch_latent_pair(c, lp, grid, st)
                          : tree ? launch_of<true>(c, lp, rows, grid, st)
                                 : launch_of<false>(c, lp, rows, grid, st);
    // a boundary that locate() leaves inside a tile lies behind its item_cost and the first key tile, and before the
    // item_slack last ones: tiles of fewer key tiles than that, and those of a single team, are never split
    if (e != cudaSuccess || p.max_kv <= (p.item_slack + 1) * kKeyTile || grid == team) return e;
    const int join = 2 * grid < max_ctas ? 2 * grid : max_ctas;
    return launch_pdl(attn_latent_join_kernel, join, kJoinThreads, 0, st, lp, grid);
}

}  // namespace moe
