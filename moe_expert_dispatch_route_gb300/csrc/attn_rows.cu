// Paged attention for query tiles of up to 32 rows (a decode step, a draft).  The keys and
// values of a request are read once and HBM bounds the work; the products run on mma.sync,
// whose fragments keep scores, probabilities and output in registers, transposed:
//   S^T = K Q^T    m = 16 keys, n = 8 rows      O^T += V^T P^T    m = 16 columns, n = 8 rows
// so that a decode step's 4 to 8 rows fill an instruction's n instead of half of its m, and o
// takes head_dim / 4 registers for every 8 rows.  Warps share out a tile's keys, each with its
// own running maximum and sum; they are put together once per query tile.
//
//   12 (or 8) consumer warps   row group x key group x tile group: kRW groups of 8 * kNT rows,
//                              kKW warps sharing a tile's keys, kTG groups taking tiles in turn
//   4 warps beside them        copies of K tiles; of V tiles; of their scales (e4m3); query rows
//                              and what else the consumers need to know of the next query tile
// A copying warp issues a copy about every 100 cycles and a tile in 16-token pages takes 8 or 16
// of them, so K and V have a warp each.
//
// An e4m3 cache is multiplied in fp16, which holds every e4m3 code exactly: one conversion
// instruction makes two codes an operand, where bf16 takes five (shifts and masks), and the
// conversions, not HBM, would bound the kernel.  What else the products need is put into fp16's
// range exactly:
//   q   a row is multiplied by a power of two that brings its largest element into [2^14, 2^15);
//       an element 2^29 below that becomes subnormal, an absolute error of 2^-40 of the largest
//   p   2^7 p 2^(s - r), s the value's scale exponent, r a reference at most 2^12 above it: at most
//       2^15, and where fp16's range ends what it adds to o is off by 2^-32 of a value at the reference
// 32 keys among which a value's scale lies elsewhere take their weights and values in bf16 (attn.cuh).
//
// The running maximum is followed loosely: o and the sum stay relative to an older maximum
// until a row's new one is 2^8 times as large (in the probabilities, which are then at most
// 2^8).  The quotient o / sum does not depend on the reference point.  With 16 rows a warp
// the exact maximum of one of them moved with almost every chunk, and o with it.
//
// Measured: 128 requests of up to 16384 bf16 tokens, 32 / 4 heads of 128, 285-289 us (6.8 TB/s); 96 of up
// to 20001 e4m3 tokens, 64 / 8 heads, 304-313 us (6.5 TB/s; with scales 2^40 apart everywhere 377); drafts of
// 30 rows over a 4096 window, 8 heads of 64, 52 us (4.2 TB/s: start, joins and the consumers' latency; e4m3
// 62); one request of 777 tokens 7.8 us, a chain of dependent loads and barriers.
#include "attn.cuh"

#include <type_traits>

namespace moe {
namespace attn {
namespace {

// What the consumers know of a query tile, in shared memory.
template <int kRows>
struct TileInfo {
    Item it;
    int stop;              // no more tiles
    int lo_all, hi_all;    // keys that every row sees: no mask there
    int2 range[kRows];     // the keys a row sees
    float row_scale[kRows];
};

template <int kD, bool kFp8, int kNT, int kRW>
struct Cfg {
    static constexpr int kElt = kFp8 ? 1 : 2;
    static constexpr int kRows = 8 * kNT * kRW;
    // Tile groups: with two stages each they overlap each other's waits; a few rows take so
    // little time that one each will do; 32 rows of wide bf16 tiles, whose ring holds three,
    // stay together on one tile.
    static constexpr bool kWide = kD * kElt == 256;
    static constexpr int kTG = kRW == 2 && kWide ? 1 : 3;
    static constexpr int kKW = kRW == 1 ? 4 : kWide ? 4 : 2;
    static constexpr int kMerged = kKW * kTG;  // key groups to be put together
    static constexpr int kWarps = kRW * kMerged;
    static constexpr int kConsumers = 32 * kWarps;
    static constexpr int kThreads = kConsumers + 128;
    static constexpr int kWarpKeys = kKeyTile / kKW;
    static constexpr int kStrips = 2;  // of 16 keys, at a time
    static constexpr int kChunks = kWarpKeys / (16 * kStrips);
    static constexpr int kTileBytes = kKeyTile * kD * kElt;  // of K or V
    static constexpr int kRowBytes = kD * kElt < 128 ? kD * kElt : 128;
    static constexpr int kHalves = kD * kElt / kRowBytes;  // 128-byte column blocks
    // stages of K and V: a multiple of kTG, so that a stage always serves the same tile group and
    // no warp's wait can miss a phase.  192 KB in flight (144 KB of the smallest) cover HBM's latency.
    static constexpr int kStages = kTileBytes == 32768 ? 3 : kTileBytes == 16384 ? 6 : 9;
    static constexpr int kRing = 2 * kStages * kTileBytes;
    static constexpr int kQStride = 2 * kD + 16;  // bytes; rows fall into different banks
    static constexpr int kOStride = kD + 4;       // floats; likewise
    static constexpr int kGroupBytes = kRows * kOStride * 4;  // o of one key group
    static constexpr int kFixed = 1024 + kRing + (kFp8 ? 2 * kStages * kKeyTile : 0) + kMerged * kRows * 8 +
                                  (4 * kStages + 8) * 8;
    static constexpr int kInfoBytes = ((int)sizeof(TileInfo<kRows>) + 15) / 16 * 16 + kRows * kQStride;
    static constexpr int kBudget = 232448 - 256;  // less the static shared memory
    // the next tile's rows are fetched ahead where there is room for them
    static constexpr int kInfos = kBudget - kFixed - 2 * kInfoBytes >= kGroupBytes ? 2 : 1;
    static constexpr int kRoom = (kBudget - kFixed - kInfos * kInfoBytes) / kGroupBytes;
    static constexpr int kSlots = kRoom < kMerged ? kRoom : kMerged;
    static constexpr int kSmem = kFixed + kInfos * kInfoBytes + kSlots * kGroupBytes;
    static_assert(kSlots >= 1 && kStages % kTG == 0, "");
    static_assert(kRing >= (kMaxRequests + 32) * 4, "locate()'s scratch");
};

// ---------------------------------------------------------------- fragments
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// An 8x8 matrix of 16-bit elements, two of a row per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (kF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
            "%1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, "
            "%1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte chunk `c` of key row `r` in a tile as TMA's swizzle left it.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    if (kRowBytes == 128) {
        const int half = c >> 3;
        return (uint32_t)(half * kKeyTile * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    }
    return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// 4 bytes global -> shared, or 4 zero bytes; and this thread's arrival on `bar` (one of those
// it counts) once its copies so far have landed.
__device__ __forceinline__ void cp_async_4_or_0(void* dst, const void* src, bool copy) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)),
                 "l"(static_cast<uint64_t>(__cvta_generic_to_global(src))), "r"(copy ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

// ---------------------------------------------------------------- query rows
// One warp: loads of the first pieces of the item's rows, 16 bytes each, all under way at once.
template <int kD, int kRows>
struct RowLoads {
    static constexpr int kPieces = kD / 8;                  // of a row
    static constexpr int kAll = kRows * kPieces / 32;       // per lane
    static constexpr int kBatch = kAll < 16 ? kAll : 16;
    uint4 x[kBatch];

    __device__ __forceinline__ void load(const Params& p, const Item& it, int i0) {
        const int rows = it.tokens * p.group;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = (i0 + b) * 32 + (threadIdx.x & 31), r = i / kPieces;
            x[b] = make_uint4(0, 0, 0, 0);
            if (r < rows) {
                const RowAt at = row_at(p, it, r);
                x[b] = __ldg(reinterpret_cast<const uint4*>(p.q + at.token * p.q_ld + at.head * p.q_head) + i % kPieces);
            }
        }
    }
};
// The same warp: the rows into `qs` (bf16 as they are; for an e4m3 cache fp16, scaled, and in the
// order in which the keys' fragments hold their columns), and what else the consumers need.
template <int kD, bool kFp8, int kRows>
__device__ void stage_rows(const Params& p, const Item& it, RowLoads<kD, kRows>& loads, TileInfo<kRows>* info,
                           uint8_t* qs, int stride) {
    using Loads = RowLoads<kD, kRows>;
    static_assert(kRows * Loads::kPieces % 32 == 0 && Loads::kAll % Loads::kBatch == 0, "");
    const int lane = threadIdx.x & 31;
    const int rows = it.tokens * p.group;
    if (lane == 0) {
        info->it = it;
        info->stop = 0;
        const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile;
        info->hi_all = p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;
        info->lo_all = p.window > 0 ? max(0, pos0 + it.tokens - p.window) : 0;
    }
    for (int r = lane; r < kRows; r += 32) {
        int2 v = make_int2(0, 0);
        if (r < rows) {
            const int pos = it.r.kv - it.r.n + it.tile * p.tokens_per_tile + r / p.group;
            v.y = p.causal ? min(pos + 1, it.r.kv) : it.r.kv;
            v.x = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        }
        info->range[r] = v;
        if (!kFp8) info->row_scale[r] = p.scale_log2;
    }
    for (int i0 = 0; i0 < Loads::kAll; i0 += Loads::kBatch) {
        if (i0 > 0) loads.load(p, it, i0);
#pragma unroll
        for (int b = 0; b < Loads::kBatch; ++b) {
            const int i = (i0 + b) * 32 + lane, r = i / Loads::kPieces, piece = i % Loads::kPieces;
            uint8_t* row = qs + r * stride;
            const uint4 x = loads.x[b];
            if (!kFp8) {
                *reinterpret_cast<uint4*>(row + piece * 16) = x;
                continue;
            }
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t mx = 0;  // largest magnitude as bf16 bits
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = __vmaxu2(mx, w[j] & 0x7fff7fffu);
            mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
            for (int o = Loads::kPieces / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const int up = f16_row_exp(mx), u1 = up / 2, u2 = up - u1;  // in two factors, each a float
            uint32_t f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = pack_f16x2(__uint_as_float(w[j] << 16) * pow2(u1) * pow2(u2),
                                  __uint_as_float(w[j] & 0xffff0000u) * pow2(u1) * pow2(u2));
            // of 16 columns, 4c and 4c + 1 stand at 2c, 4c + 2 and 4c + 3 at 8 + 2c
            uint8_t* at = row + (piece >> 1) * 32 + (piece & 1) * 8;
            *reinterpret_cast<uint2*>(at) = make_uint2(f[0], f[2]);
            *reinterpret_cast<uint2*>(at + 16) = make_uint2(f[1], f[3]);
            // not 0: a row whose scores are all but 0 must not make -inf * 0 of the mask
            if (piece == 0) info->row_scale[r] = fmaxf(p.scale_log2 * pow2(-u1) * pow2(-u2), 0x1p-149f);
        }
    }
}

// The output rows of a split tile from its parts, in CTA order: a thread takes four columns of a
// row, the loads of eight parts under way together (a long context is split over the whole GPU).
template <int kD, int kThreads>
__device__ void join_rows(const Params& p, const Item& it, const Parts& parts, int rows) {
    constexpr int kPer = kD / 4, kBatch = 8;
    for (int r = threadIdx.x / kPer; r < rows; r += kThreads / kPer) {
        const int d = (threadIdx.x % kPer) * 4;
        float m = -CUDART_INF_F, l = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b0 = parts.first; b0 <= parts.last; b0 += kBatch) {
            float2 ml[kBatch];
            float4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int c = b0 + i, slot = part_slot(parts, c);
                ml[i] = make_float2(-CUDART_INF_F, 0.0f);
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c <= parts.last) {
                    ml[i] = __ldcg(part_ml(p, c, slot) + r);
                    x[i] = __ldcg(reinterpret_cast<const float4*>(part_o(p, c, slot) + (size_t)r * kD + d));
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float mn = fmaxf(m, ml[i].x);
                const float base = mn == -CUDART_INF_F ? 0.0f : mn;
                const float fa = exp2_fast(m - base), fb = exp2_fast(ml[i].x - base);
                l = l * fa + ml[i].y * fb;
                o.x = o.x * fa + x[i].x * fb;
                o.y = o.y * fa + x[i].y * fb;
                o.z = o.z * fa + x[i].z * fb;
                o.w = o.w * fa + x[i].w * fb;
                m = mn;
            }
        }
        const RowAt at = row_at(p, it, r);
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        *reinterpret_cast<uint2*>(p.o + at.token * p.o_ld + at.head * p.o_head + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (p.lse && d == 0)
            p.lse[(int64_t)at.token * p.heads * p.group + at.head] =
                l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <int kD, bool kFp8, int kNT, int kRW>
__global__ void __launch_bounds__(Cfg<kD, kFp8, kNT, kRW>::kThreads, 1)
    attn_rows_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const uint8_t* __restrict__ k_scale,
                     const uint8_t* __restrict__ v_scale) {
    using C = Cfg<kD, kFp8, kNT, kRW>;
    using Info = TileInfo<C::kRows>;
    constexpr int kSteps = kD / 16;  // k-steps of the first product, column tiles of the second
    extern __shared__ uint8_t smem_raw[];
    // aligned by an offset, so that accesses stay in the shared window with 32-bit addresses
    uint8_t* ring = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);
    float* xchg = reinterpret_cast<float*>(ring + C::kRing);  // o of kSlots key groups
    uint8_t* infos = reinterpret_cast<uint8_t*>(xchg) + C::kSlots * C::kGroupBytes;
    uint8_t* scales = infos + C::kInfos * C::kInfoBytes;
    float2* group_ml = reinterpret_cast<float2*>(scales + (kFp8 ? 2 * C::kStages * kKeyTile : 0));
    uint64_t* full = reinterpret_cast<uint64_t*>(group_ml + C::kMerged * C::kRows);  // [stage][K, V]
    uint64_t* empty = full + 2 * C::kStages;
    uint64_t* info_full = empty + 2 * C::kStages;
    uint64_t* info_empty = info_full + 2;
    uint64_t* never = info_empty + 2;
    __shared__ Start start;
    __shared__ int abort_s, last_s;
    volatile int* abort = &abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int i = 0; i < 2 * C::kStages; ++i) {
            tc::mbar_init(&full[i], kFp8 ? 33 : 1);
            tc::mbar_init(&empty[i], kRW * C::kKW);
        }
        for (int i = 0; i < C::kInfos; ++i) {
            tc::mbar_init(&info_full[i], 32);
            tc::mbar_init(&info_empty[i], 1);
        }
        tc::mbar_init(never, 1);
        tc::fence_barrier_init();
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    __syncthreads();
    pdl_begin();
    locate<C::kThreads>(p, reinterpret_cast<uint32_t*>(ring), &start);
    // one thread: counts a part that this CTA gives up, as if it had been stored
    auto let_go = [&](const Item& it) {
        if (it.whole) return;
        const Parts parts = parts_of(p, it, start);
        int last;
        last_of(p.counters + parts.last, parts.last - parts.first + 1, 0, &last, [] {});
    };
    if (p.inject_ns > 0 && blockIdx.x == 0) {  // test hook: the failure path of a bounded wait
        if (threadIdx.x == 0) {
            tc::wait_on_nothing(never, (uint64_t)p.inject_ns);
            set_err(p.err, MOE_ERR_TIMEOUT);
            for (Cursor cur = cursor(start); more(cur);) let_go(take(p, cur));
        }
        return;
    }
    // a wait that runs out is reported and then passed, here and in every later wait, so that
    // each barrier is still met; the results are void
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!tc::mbar_wait(bar, parity, abort)) {
            set_err(p.err, MOE_ERR_TIMEOUT);
            *abort = 1;
        }
        __syncwarp();
    };

    if (warp >= C::kWarps) {
        Cursor cur = cursor(start);
        const int role = warp - C::kWarps;  // 0: K, 1: V, 2: scales, 3: query rows
        if (role == 3) {
            uint32_t n = 0;
            for (bool stop = false; !stop; ++n) {
                const int buf = n % C::kInfos;
                uint8_t* at = infos + buf * C::kInfoBytes;
                Info* info = reinterpret_cast<Info*>(at);
                stop = !more(cur);
                Item it;
                RowLoads<kD, C::kRows> loads;
                if (!stop) {
                    it = take(p, cur);
                    loads.load(p, it, 0);
                }
                // not cut short by an abort: the consumers meet for every query tile
                if (n >= C::kInfos && !tc::mbar_wait_bounded(&info_empty[buf], (n / C::kInfos - 1) & 1)) {
                    // the consumers are told that there is no more, and the parts left are counted
                    set_err(p.err, MOE_ERR_TIMEOUT);
                    *abort = 1;
                    if (lane == 0) {
                        if (!stop) let_go(it);
                        while (more(cur)) let_go(take(p, cur));
                    }
                    stop = true;
                }
                __syncwarp();
                if (stop) {
                    if (lane == 0) info->stop = 1;
                } else {
                    stage_rows<kD, kFp8, C::kRows>(p, it, loads, info, at + C::kInfoBytes - C::kRows * C::kQStride,
                                                   C::kQStride);
                }
                tc::mbar_arrive(&info_full[buf]);
            }
            return;
        }
        if (role == 2) {
            // scales: four keys of K and of V a lane, each 4-byte copy signalling the stage's barrier
            // itself (as bulk copies they were 16 bytes each for 16-token pages, as many as of tiles' boxes)
            if (!kFp8) return;
            int stage = 0;
            uint32_t turn = 0;
            while (more(cur)) {
                const Item it = take(p, cur);
                Pages pages = pages_of(p, it);
                for (int k = 0; k < it.n; ++k) {
                    const int key0 = (it.k0 + k) * kKeyTile, key = key0 + lane * 4;
                    const int page = page_of(p, it, pages, key0, (key >> p.page_shift) - (key0 >> p.page_shift));
                    const bool want = key < it.s.hi && key + 4 > it.s.lo && page >= 0 && page < p.num_pages;
                    const int64_t at =
                        want ? ((int64_t)page * p.heads + it.head) * p.page_size + (key & (p.page_size - 1)) : 0;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (turn > 0) wait(&empty[2 * stage + kv], (turn - 1) & 1);
                        cp_async_4_or_0(scales + (2 * stage + kv) * kKeyTile + lane * 4, (kv ? v_scale : k_scale) + at,
                                        want);
                        cp_async_arrive(&full[2 * stage + kv]);
                    }
                    if (++stage == C::kStages) stage = 0, ++turn;
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            return;
        }
        const int box_keys = min(p.page_size, kKeyTile), npg = kKeyTile / box_keys;
        int stage = 0;
        uint32_t turn = 0, sent = 0;
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
            if (it.n == 0) ahead();
            for (int k = 0; k < it.n; ++k) {
                const int key0 = (it.k0 + k) * kKeyTile;
                // lane i copies box i of the tile (page i / kHalves of it, column block i % kHalves)
                const int pg = lane / C::kHalves, part = lane % C::kHalves;
                const int key = key0 + pg * box_keys, off = key & (p.page_size - 1);
                const bool want = pg < npg && key < it.s.hi && key + box_keys > it.s.lo;
                int page = page_of(p, it, pages, key0, pg);
                if (want && (page < 0 || page >= p.num_pages)) {
                    set_err(p.err, MOE_ERR_BAD_INDEX);
                    page = p.num_pages;  // past the pool: the copy fills zeros
                }
                uint64_t* bar = &full[2 * stage + role];
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, want)) * (box_keys * C::kRowBytes);
                if (turn > 0) wait(&empty[2 * stage + role], (turn - 1) & 1);
                if (!*abort) {
                    ++sent;
                    if (lane == 0) tc::mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    if (want)
                        tc::tma_load_4d(ring + (2 * stage + role) * C::kTileBytes +
                                            (part * kKeyTile + pg * box_keys) * C::kRowBytes,
                                        role ? &vmap : &kmap, bar, part * (C::kRowBytes / C::kElt), off, it.head, page);
                }
                if (++stage == C::kStages) stage = 0, ++turn;
                if (k == 0) ahead();
            }
        }
        if (*abort)  // copies still in flight land (or a bounded wait gives up) before the CTA ends
            for (int i = 0; i < C::kStages; ++i) {
                const uint32_t times = (sent + C::kStages - 1 - i) / C::kStages;  // that stage i has been copied to
                if (times > 0) tc::mbar_wait_bounded(&full[2 * i + role], (times - 1) & 1);
            }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int rg = warp % kRW, mg = warp / kRW, kg = mg % C::kKW, tg = mg / C::kKW;
    const int g = lane >> 2, c = lane & 3;
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(C::kConsumers) : "memory"); };
    uint32_t tiles = 0;  // key tiles of the query tiles so far
    for (uint32_t n = 0;; ++n) {
        const int buf = n % C::kInfos;
        const Info* info = reinterpret_cast<const Info*>(infos + buf * C::kInfoBytes);
        const uint32_t q_addr = tc::smem_u32(info) + C::kInfoBytes - C::kRows * C::kQStride + rg * 8 * kNT * C::kQStride;
        // (twice as long as the warp that fills it may wait before it says that there is no more)
        if (!tc::mbar_wait_bounded(&info_full[buf], (n / C::kInfos) & 1) &&
            !tc::mbar_wait_bounded(&info_full[buf], (n / C::kInfos) & 1)) {
            set_err(p.err, MOE_ERR_TIMEOUT);
            *abort = 1;
            return;  // every consumer waits here, and none past it
        }
        __syncwarp();
        if (info->stop) return;
        float o[kSteps][kNT][4];
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][t][i] = 0.0f;
        // this thread's rows are 8 t + 2 c + x of the row group; m is before row_scale (> 0)
        float m[kNT][2], l[kNT][2], base[kNT][2], row_scale[kNT][2];
        int2 range[kNT][2];
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = rg * 8 * kNT + t * 8 + c * 2 + x;
                m[t][x] = -CUDART_INF_F;
                l[t][x] = base[t][x] = 0.0f;
                row_scale[t][x] = info->row_scale[r];
                range[t][x] = info->range[r];
            }
        const int lo_all = info->lo_all, hi_all = info->hi_all, lo_any = info->it.s.lo, hi_any = info->it.s.hi;
        const int tile0 = info->it.k0, count = info->it.n;
        Scales vs = {0, 0, 0, 0};  // e4m3: of the values
        for (int kt = (tg + C::kTG - (int)(tiles % C::kTG)) % C::kTG; kt < count; kt += C::kTG) {
            const uint32_t at = tiles + kt, stage = at % C::kStages, parity = (at / C::kStages) & 1;
            const uint32_t k_addr = tc::smem_u32(ring + 2 * stage * C::kTileBytes), v_addr = k_addr + C::kTileBytes;
            const uint8_t* sc_at = scales + 2 * stage * kKeyTile;
            wait(&full[2 * stage], parity);
#pragma unroll 1
            for (int ch = 0; ch < C::kChunks; ++ch) {
                const int in0 = kg * C::kWarpKeys + ch * 16 * C::kStrips;  // first key within the tile
                const int key0 = (tile0 + kt) * kKeyTile + in0;
                const bool edge = key0 < lo_all || key0 + 16 * C::kStrips > hi_all;
                // ---- scores: element (key g + 8 (i / 2), row 2 c + i % 2)
                float s[C::kStrips][kNT][4];
#pragma unroll
                for (int st = 0; st < C::kStrips; ++st)
#pragma unroll
                    for (int t = 0; t < kNT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[st][t][i] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < kSteps; ks += 2) {
                    uint32_t q[kNT][4];  // two k-steps
#pragma unroll
                    for (int t = 0; t < kNT; ++t)
                        ldsm_x4(q[t], q_addr + (t * 8 + (lane & 7)) * C::kQStride + (2 * ks + (lane >> 3)) * 16);
#pragma unroll
                    for (int st = 0; st < C::kStrips; ++st) {
                        const int row0 = in0 + st * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
                        uint32_t a[2][4];
                        if (kFp8) {
                            uint32_t w[4];  // keys 0-7 and 8-15 of chunk ks, then of chunk ks + 1
                            ldsm_x4(w, k_addr + swizzled<C::kRowBytes>(row0, ks + (lane >> 4)));
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                e4m3x4_f16(w[2 * u], a[u][0], a[u][2]);
                                e4m3x4_f16(w[2 * u + 1], a[u][1], a[u][3]);
                            }
                        } else {
                            ldsm_x4(a[0], k_addr + swizzled<C::kRowBytes>(row0, 2 * ks + (lane >> 4)));
                            ldsm_x4(a[1], k_addr + swizzled<C::kRowBytes>(row0, 2 * ks + 2 + (lane >> 4)));
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int t = 0; t < kNT; ++t) mma16816<kFp8>(s[st][t], a[u], q[t][2 * u], q[t][2 * u + 1]);
                    }
                }
                // ---- the keys' scales, the mask, the running maximum
                const float kscale = kFp8 ? scale_of(sc_at[in0 + lane]) : 1.0f;  // lane i: key i's
                float mx[kNT][2];
#pragma unroll
                for (int t = 0; t < kNT; ++t) mx[t][0] = mx[t][1] = -CUDART_INF_F;
#pragma unroll
                for (int st = 0; st < C::kStrips; ++st)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float f = kFp8 ? __shfl_sync(0xffffffffu, kscale, st * 16 + y * 8 + g) : 1.0f;
                        const int key = key0 + st * 16 + y * 8 + g;
#pragma unroll
                        for (int t = 0; t < kNT; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                float v = s[st][t][2 * y + x];
                                if (kFp8) v *= f;
                                if (edge && (key < range[t][x].x || key >= range[t][x].y)) v = -CUDART_INF_F;
                                s[st][t][2 * y + x] = v;
                                mx[t][x] = fmaxf(mx[t][x], v);
                            }
                    }
                if (ch == C::kChunks - 1) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&empty[2 * stage]);
                }
                bool up = false;
#pragma unroll
                for (int t = 0; t < kNT; ++t)
                    up |= (mx[t][0] - m[t][0]) * row_scale[t][0] > kLoose ||  // also from -inf
                          (mx[t][1] - m[t][1]) * row_scale[t][1] > kLoose;
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int t = 0; t < kNT; ++t)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1)
                                mx[t][x] = fmaxf(mx[t][x], __shfl_xor_sync(0xffffffffu, mx[t][x], w));
                            const float mn = fmaxf(m[t][x], mx[t][x]);
                            const float f =
                                m[t][x] == -CUDART_INF_F ? 0.0f : exp2_fast((m[t][x] - mn) * row_scale[t][x]);
                            m[t][x] = mn;
                            base[t][x] = mn == -CUDART_INF_F ? 0.0f : -mn * row_scale[t][x];
                            l[t][x] *= f;
#pragma unroll
                            for (int j = 0; j < kSteps; ++j) {
                                o[j][t][x] *= f;
                                o[j][t][2 + x] *= f;
                            }
                        }
                }
                // ---- probabilities
                if (ch == 0) wait(&full[2 * stage + 1], parity);
                // keys of this chunk that no row sees hold anything, NaN among it: their values read as 0
                const bool tail = key0 < lo_any || key0 + 16 * C::kStrips > hi_any;
                float vscale = 1.0f;  // e4m3: of key `lane`
                bool far = false;
                if (kFp8) {
                    const bool unseen = tail && (key0 + lane < lo_any || key0 + lane >= hi_any);
                    uint32_t vb = sc_at[kKeyTile + in0 + lane];
                    if (unseen) vb = vs.ref;  // its value reads as 0
                    vscale = __uint_as_float((vb - vs.ref + kPBits + 127) << 23);
                    if (__any_sync(0xffffffffu, vs.ref - vb > vs.span)) {
                        const bool counts = !unseen && vb < 255;
                        const uint32_t lo = __reduce_min_sync(0xffffffffu, counts ? vb : 255u);
                        const uint32_t top = __reduce_max_sync(0xffffffffu, counts ? vb : 0u), was = vs.ref;
                        take_in(vs, lo, top);
                        if (vs.ref != was) {
                            const float f = pow2((int)was - (int)vs.ref);
#pragma unroll
                            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                                for (int t = 0; t < kNT; ++t)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) o[j][t][i] *= f;
                        }
                        if (unseen) vb = vs.ref;
                        far = !near_ref(vs, min(lo, top), top);
                        vscale = vb == 255 ? CUDART_NAN_F : pow2((int)vb - (int)vs.ref + kPBits);
                    }
                }
                auto weigh = [&](auto far_t) {
                    constexpr bool kFar = decltype(far_t)::value;  // e4m3: weights and values in bf16
                    uint32_t pb[C::kStrips][kNT][2];  // (row g, keys 2c, 2c + 1) and 8 keys further
#pragma unroll
                    for (int st = 0; st < C::kStrips; ++st)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float f = kFp8 ? __shfl_sync(0xffffffffu, vscale, st * 16 + y * 8 + g) : 1.0f;
#pragma unroll
                            for (int t = 0; t < kNT; ++t) {
                                const float p0 = exp2_fast(fmaf(s[st][t][2 * y], row_scale[t][0], base[t][0]));
                                const float p1 = exp2_fast(fmaf(s[st][t][2 * y + 1], row_scale[t][1], base[t][1]));
                                l[t][0] += p0;
                                l[t][1] += p1;
                                pb[st][t][y] = transpose8(!kFp8  ? pack_bf16x2(p0, p1)
                                                          : kFar ? pack_bf16x2(p0 * f, p1 * f)
                                                                 : pack_f16x2(p0 * f, p1 * f));
                            }
                        }
                    // ---- o += p v
#pragma unroll
                    for (int st = 0; st < C::kStrips; ++st) {
                        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of the key pairs 2c, 2c + 1 and 8 further
                        if (tail) {
#pragma unroll
                            for (int y = 0; y < 2; ++y)
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const int key = key0 + st * 16 + y * 8 + c * 2 + x;
                                    if (key < lo_any || key >= hi_any) keep[y] &= x ? 0x0000ffffu : 0xffff0000u;
                                }
                        }
                        if (kFp8) {
#pragma unroll
                            for (int j = 0; j < kSteps; j += 2) {
                                uint32_t w[4];  // keys 0-7 and 8-15 of chunk j, then of chunk j + 1
                                ldsm_x4_t(w, v_addr + swizzled<C::kRowBytes>(
                                                          in0 + st * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), j + (lane >> 4)));
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    // bytes: a pair of keys of column 2 g, then of column 2 g + 1
                                    uint32_t w0 = __byte_perm(w[2 * u], 0, 0x3120);
                                    uint32_t w1 = __byte_perm(w[2 * u + 1], 0, 0x3120);
                                    if (tail) {
                                        w0 &= __byte_perm(keep[0], 0, 0x2020);
                                        w1 &= __byte_perm(keep[1], 0, 0x2020);
                                    }
                                    uint32_t a[4];
                                    e4m3x4_f16(w0, a[0], a[1]);
                                    e4m3x4_f16(w1, a[2], a[3]);
                                    if (kFar) {
#pragma unroll
                                        for (int i = 0; i < 4; ++i) a[i] = f16x2_bf16x2(a[i]);
                                    }
#pragma unroll
                                    for (int t = 0; t < kNT; ++t)
                                        mma16816<!kFar>(o[j + u][t], a, pb[st][t][0], pb[st][t][1]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < kSteps; ++j) {
                                uint32_t a[4];
                                ldsm_x4_t(a, v_addr + swizzled<C::kRowBytes>(in0 + st * 16 + (lane >> 4) * 8 + (lane & 7),
                                                                             2 * j + ((lane >> 3) & 1)));
                                if (tail) a[0] &= keep[0], a[1] &= keep[0], a[2] &= keep[1], a[3] &= keep[1];
#pragma unroll
                                for (int t = 0; t < kNT; ++t) mma16816<false>(o[j][t], a, pb[st][t][0], pb[st][t][1]);
                            }
                        }
                    }
                };
                if (kFp8 && far)
                    weigh(std::true_type{});
                else
                    weigh(std::false_type{});
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[2 * stage + 1]);
        }

        // ---- put the key groups that had keys together, relative to the rows' common maximum, in a
        // fixed order.  rank: place of this warp's group among them
        const int rank = (tg + C::kTG - (int)(tiles % C::kTG)) % C::kTG * C::kKW + kg;
        const int groups = min(count, C::kTG) * C::kKW;
        tiles += count;
        if (rank < groups) {
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    m[t][x] *= row_scale[t][x];  // in powers of two
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) l[t][x] += __shfl_xor_sync(0xffffffffu, l[t][x], w);
                }
            if (kFp8) {  // back from 2^7 2^-r, and relative to a maximum that keeps the sums of o in range
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int up = sum_exp(l[t][x]), e2 = (int)vs.ref - 127 - kPBits - up;
                        const float f1 = pow2(e2 / 2), f2 = pow2(e2 - e2 / 2);
                        m[t][x] += (float)up;
                        l[t][x] *= pow2(-up);
#pragma unroll
                        for (int j = 0; j < kSteps; ++j)
#pragma unroll
                            for (int i = x; i < 4; i += 2) o[j][t][i] = o[j][t][i] * f1 * f2;
                    }
            }
        }
        // where an element stands: column 16 j + g (+ 8), or 16 j + 2 g (+ 1) from e4m3 pairs
        constexpr int kColG = kFp8 ? 2 : 1, kColHi = kFp8 ? 1 : 8;
        float* mine =
            xchg + (rank % C::kSlots) * (C::kRows * C::kOStride) + (rg * 8 * kNT + c * 2) * C::kOStride + g * kColG;
        float2* mine_ml = group_ml + (rank % C::kSlots) * C::kRows + rg * 8 * kNT + c * 2;
        auto put = [&] {
#pragma unroll
            for (int t = 0; t < kNT; ++t) {
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mine[(t * 8 + (i & 1)) * C::kOStride + j * 16 + (i >> 1) * kColHi] = o[j][t][i];
                if (g == 0) {
                    mine_ml[t * 8] = make_float2(m[t][0], l[t][0]);
                    mine_ml[t * 8 + 1] = make_float2(m[t][1], l[t][1]);
                }
            }
        };
        // kSlots groups at a time hand their state to the first kSlots
        for (int b = (groups - 1) / C::kSlots * C::kSlots; b > 0; b -= C::kSlots) {
            if (rank >= b && rank < b + C::kSlots && rank < groups) put();
            sync();
            if (rank < C::kSlots && rank + b < groups) {
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 ml = mine_ml[t * 8 + x];
                        const float mn = fmaxf(m[t][x], ml.x), to = mn == -CUDART_INF_F ? 0.0f : mn;
                        const float fa = exp2_fast(m[t][x] - to), fb = exp2_fast(ml.x - to);
                        m[t][x] = mn;
                        l[t][x] = l[t][x] * fa + ml.y * fb;
#pragma unroll
                        for (int j = 0; j < kSteps; ++j)
#pragma unroll
                            for (int i = x; i < 4; i += 2)
                                o[j][t][i] = o[j][t][i] * fa +
                                             mine[(t * 8 + x) * C::kOStride + j * 16 + (i >> 1) * kColHi] * fb;
                    }
            }
            sync();
        }
        const int left = min(groups, C::kSlots);
        if (rank < left) put();
        sync();
        const Item& it = info->it;
        const int rows = it.tokens * p.group;
        for (int i = threadIdx.x; i < rows * (kD / 4); i += C::kConsumers) {
            const int r = i / (kD / 4), d = (i % (kD / 4)) * 4;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            float2 ml = make_float2(-CUDART_INF_F, 0.0f);
#pragma unroll
            for (int k = 0; k < C::kSlots; ++k)
                if (k < left) ml.x = fmaxf(ml.x, group_ml[k * C::kRows + r].x);
            const float to = ml.x == -CUDART_INF_F ? 0.0f : ml.x;
#pragma unroll
            for (int k = 0; k < C::kSlots; ++k)
                if (k < left) {
                    const float2 other = group_ml[k * C::kRows + r];
                    const float f = exp2_fast(other.x - to);
                    const float4 v = *reinterpret_cast<const float4*>(xchg + (k * C::kRows + r) * C::kOStride + d);
                    ml.y += other.y * f;
                    a.x += v.x * f, a.y += v.y * f, a.z += v.z * f, a.w += v.w * f;
                }
            if (it.whole) {
                const RowAt at = row_at(p, it, r);
                const float inv = ml.y > 0.0f ? 1.0f / ml.y : (ml.y == 0.0f ? 0.0f : ml.y);
                *reinterpret_cast<uint2*>(p.o + at.token * p.o_ld + at.head * p.o_head + d) =
                    make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
                if (p.lse && d == 0)
                    p.lse[(int64_t)at.token * p.heads * p.group + at.head] =
                        ml.y == 0.0f ? -CUDART_INF_F : (ml.x + log2f(ml.y)) * 0.6931471805599453f;
            } else {
                const int slot = it.first ? 0 : 1;
                *reinterpret_cast<float4*>(part_o(p, blockIdx.x, slot) + (size_t)r * kD + d) = a;
                if (d == 0) part_ml(p, blockIdx.x, slot)[r] = ml;
            }
        }
        if (!it.whole) {
            const Parts parts = parts_of(p, it, start);
            if (last_of(p.counters + parts.last, parts.last - parts.first + 1, threadIdx.x, &last_s, sync))
                join_rows<kD, C::kConsumers>(p, it, parts, rows);
        }
        sync();
        if (threadIdx.x == 0) tc::mbar_arrive(&info_empty[buf]);
    }
}

template <int kD, bool kFp8, int kNT, int kRW>
cudaError_t launch_as(const moe_kv_cache& c, Params& p, int grid_cap, cudaStream_t st) {
    using C = Cfg<kD, kFp8, kNT, kRW>;
    p.tokens_per_tile = C::kRows / p.group;
    // what a query tile costs beside its key tiles is about 3 us, a K and V tile 1.5 us per 64 KB
    p.item_cost = 2 * 32768 / C::kTileBytes;
    p.item_slack = 1;
    // runs of at least 2 units: one request of 4000 tokens 8.8 us, with runs of 1 9.9 and of 3 9.0 (32 rows
    // over 2000: 15.2, 17.8 and 15.9; 777 tokens 7.8, 7.5 and 7.8)
    p.cta_units = 2;
    CUtensorMap km, vm;
    if (!make_pool_map(&km, c, c.k) || !make_pool_map(&vm, c, c.v)) return cudaErrorInvalidValue;
    auto kern = attn_rows_kernel<kD, kFp8, kNT, kRW>;
    cudaError_t e = ensure_max_dynamic_smem(kern, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid_for(p, grid_cap), C::kThreads, C::kSmem, st, p, km, vm, c.k_scale, c.v_scale);
}

template <int kD, bool kFp8>
cudaError_t launch_rows_as(const moe_kv_cache& c, Params& p, int rows, int grid_cap, cudaStream_t st) {
    if (rows <= 8) return launch_as<kD, kFp8, 1, 1>(c, p, grid_cap, st);
    if (rows <= 16) return launch_as<kD, kFp8, 2, 1>(c, p, grid_cap, st);
    return launch_as<kD, kFp8, 2, 2>(c, p, grid_cap, st);
}

}  // namespace

cudaError_t launch_rows(const moe_kv_cache& c, Params& p, int rows, int grid_cap, cudaStream_t st) {
    const bool fp8 = c.dtype == MOE_FP8_E4M3;
    if (c.head_dim == 128)
        return fp8 ? launch_rows_as<128, true>(c, p, rows, grid_cap, st)
                   : launch_rows_as<128, false>(c, p, rows, grid_cap, st);
    return fp8 ? launch_rows_as<64, true>(c, p, rows, grid_cap, st)
               : launch_rows_as<64, false>(c, p, rows, grid_cap, st);
}

}  // namespace attn
}  // namespace moe
