// Paged attention for query tiles of up to 64 rows (a decode step, a draft): the keys and
// values of a request are read once and HBM bounds the kernel, so the products run on
// mma.sync, whose fragments keep scores, probabilities and output in registers, and the
// warps of a CTA share out the keys of a tile instead of padding the rows to 128.
//
//   warps 8-    TMA copies of 128-key K and V tiles, page by page, into a ring
//   warps 0-7   row group = warp % kRowWarps (16 rows each), key group = warp / kRowWarps;
//               each keeps a running maximum and sum over its own keys; the key groups are
//               merged in shared memory once per query tile
//
// An e4m3 cache is multiplied in fp16, which holds every e4m3 code exactly, so a conversion
// instruction turns two codes into an operand; bf16 operands took five (shifts and masks), and
// the ALU pipe, not HBM, bounded the kernel (48 % busy at 47 % of the copy rate; 64 / 8 heads
// of 128, 96 requests: 643 us).  What else the products need is put in fp16's range exactly:
//   q   a row is multiplied by a power of two that brings its largest element into [2^14, 2^15);
//       an element 2^29 below that becomes subnormal, an absolute error of 2^-40 of the largest
//   p   2^14 p 2^(s - r), s the value's scale exponent, r the largest s so far: at most 2^14, and
//       what falls below fp16's range is under 2^-38 of the largest weight a key can have
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kConsumers = 256;
constexpr int kXchgBytes = 4 * 16 * 128 * 4;  // o of four warps

template <int kD, bool kFp8>
struct Cfg {
    static constexpr int kElt = kFp8 ? 1 : 2;
    static constexpr int kEntryBytes = kKeyTile * kD * kElt;
    static constexpr int kRowBytes = kD * kElt < 128 ? kD * kElt : 128;  // of one swizzled row
    static constexpr int kHalves = kD * kElt / kRowBytes;
    static constexpr int kEntries = kD == 64 ? 12 : kFp8 ? 8 : 6;
    // Copying warps: a warp issues a copy about every 100 cycles, and small pages make many of
    // them.  Entry i of the stream belongs to warp i % kCopyWarps, and a ring slot always to
    // the same warp, so that no warp's wait can miss a phase.
    static constexpr int kCopyWarps = kEntries % 4 == 0 ? 4 : 2;
    static constexpr int kThreads = kConsumers + 32 * kCopyWarps;
    static constexpr int kScratchBytes = (kMaxRequests + 32) * 4;  // locate(); the exchange area later
    static_assert(kScratchBytes >= kXchgBytes, "");
    static constexpr int kScaleBytes = kFp8 ? kEntries * kKeyTile : 0;
    static constexpr int kSmem = 1024 + kEntries * kEntryBytes + kScratchBytes + kScaleBytes + 4 * 16 * 8 + 512;
    static_assert(kSmem <= 232448, "");
};

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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 codes as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// 2^e as a float, 0 below its range.
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.0f : __int_as_float((min(e, 127) + 127) << 23); }

// Byte offset of 16-byte chunk `c` of key row `r` in a tile as TMA's swizzle left it.
template <int kRowBytes>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    if (kRowBytes == 128) {
        const int half = c >> 3;
        return (uint32_t)(half * kKeyTile * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    }
    return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int kD, bool kFp8, int kRowWarps>
__global__ void __launch_bounds__(Cfg<kD, kFp8>::kThreads, 1)
    attn_rows_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const uint8_t* __restrict__ k_scale,
                     const uint8_t* __restrict__ v_scale) {
    using C = Cfg<kD, kFp8>;
    // With one row warp, two groups of four warps take alternate key tiles: 32 keys a warp at a
    // time instead of 16 halve what a step costs beside its products.  A ring entry always goes
    // to the same group (whole tiles in the ring: an even number), so that no warp's wait can
    // miss a phase; the bf16 ring of head_dim 128 holds three tiles and stays with one group.
    constexpr int kTileGroups = kRowWarps == 1 && C::kEntries / 2 % 2 == 0 ? 2 : 1;
    constexpr int kKeyWarps = 8 / kRowWarps / kTileGroups;  // warps sharing a tile's keys
    constexpr int kMerged = kKeyWarps * kTileGroups;        // key groups of a query row
    constexpr int kWarpKeys = kKeyTile / kKeyWarps;
    constexpr int kStrips = kWarpKeys >= 32 ? 2 : 1;        // 16 keys each, at a time
    constexpr int kChunks = kWarpKeys / (16 * kStrips);
    constexpr int kSteps = kD / 16;  // k-steps of the first product, column pairs of the second
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* xchg = ring + C::kEntries * C::kEntryBytes;
    uint8_t* scales = xchg + C::kScratchBytes;
    float2* xml = reinterpret_cast<float2*>(scales + C::kScaleBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(xml + 4 * 16);
    uint64_t* empty = full + C::kEntries;
    uint64_t* never = empty + C::kEntries;
    __shared__ Start start;
    __shared__ int abort_s, last_s;
    volatile int* abort = &abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int i = 0; i < C::kEntries; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 8 / kTileGroups);
        }
        tc::mbar_init(never, 1);
        tc::fence_barrier_init();
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    __syncthreads();
    pdl_begin();
    if (p.inject_ns > 0) {  // test hook: the failure path of a bounded wait
        if (threadIdx.x == 0) {
            tc::wait_on_nothing(never, (uint64_t)p.inject_ns);
            set_err(p.err, MOE_ERR_TIMEOUT);
        }
        return;
    }
    locate<C::kThreads>(p, reinterpret_cast<uint32_t*>(xchg), &start);
    Cursor cur = cursor(p, start);
    if (!more(cur)) return;

    if (warp >= 8) {
        // ------------------------------------------------------------ copies
        int e = 0;
        uint32_t turn = 0, entry = 0;  // of the stream K, V, K, V, ...
        const int box_keys = min(p.page_size, kKeyTile), npg = kKeyTile / box_keys;
        auto next = [&] {
            if (++e == C::kEntries) e = 0, ++turn;
        };
        bool more_now = true;
        Item it = take(p, cur);
        Pages pages = pages_of(p, it);
        while (more_now) {
            const bool more_then = more(cur);
            Item after;
            Pages pages_after;
            if (more_then) {
                after = take(p, cur);
                pages_after = pages_of(p, after);
            }
            for (int k = 0; k < it.n; ++k) {
                const int key0 = (it.k0 + k) * kKeyTile;
                // lane i: box i of the tile (page i / kHalves of it, column half i % kHalves)
                const int pg = lane / C::kHalves, half = lane % C::kHalves;
                const int key = key0 + pg * box_keys;
                const bool want = pg < npg && key < it.s.hi && key + box_keys > it.s.lo;
                int page = page_of(p, it, pages, key0, pg);
                if (want && (page < 0 || page >= p.num_pages)) {
                    set_err(p.err, MOE_ERR_BAD_INDEX);
                    page = p.num_pages;  // past the pool: the copy fills zeros
                }
                const bool scaled = kFp8 && want && half == 0 && page < p.num_pages;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, want)) * (box_keys * C::kRowBytes) +
                                       __popc(__ballot_sync(0xffffffffu, scaled)) * box_keys;
                const int off = key & (p.page_size - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, next()) {
                    if ((int)(entry++ % C::kCopyWarps) != warp - 8) continue;
                    if (turn > 0 && !tc::mbar_wait(&empty[e], (turn - 1) & 1, abort)) {
                        if (lane == 0) set_err(p.err, MOE_ERR_TIMEOUT);
                        *abort = 1;
                    }
                    if (!*abort) {
                        if (lane == 0) tc::mbar_arrive_expect_tx(&full[e], bytes);
                        __syncwarp();
                        uint8_t* dst = ring + e * C::kEntryBytes + half * kKeyTile * C::kRowBytes +
                                       pg * box_keys * C::kRowBytes;
                        if (want)
                            tc::tma_load_4d(dst, kv ? &vmap : &kmap, &full[e], half * (C::kRowBytes / C::kElt), off, it.head,
                                        page);
                        if (scaled)
                            tc::bulk_load(scales + e * kKeyTile + pg * box_keys,
                                          (kv ? v_scale : k_scale) + ((int64_t)page * p.heads + it.head) * p.page_size +
                                              off,
                                          box_keys, &full[e]);
                    }
                }
            }
            it = after;
            pages = pages_after;
            more_now = more_then;
        }
        if (*abort)  // copies still in flight land (or a bounded wait gives up) before the CTA ends
            for (int i = warp - 8; i < C::kEntries; i += C::kCopyWarps) {
                const uint32_t issued = turn + (i < e ? 1 : 0);
                if (issued > 0) tc::mbar_wait_bounded(&full[i], (issued - 1) & 1);
            }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int rg = warp % kRowWarps, kg = warp / kRowWarps % kKeyWarps, tg = warp / kRowWarps / kKeyWarps;
    const int mg = warp / kRowWarps;  // key group among those that are merged
    uint32_t tiles = 0;               // key tiles so far
    const int g = lane >> 2, c = lane & 3;  // fragment row and column
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); };
    int e = 0;
    uint32_t turn = 0;
    auto next = [&] {
        if (++e == C::kEntries) e = 0, ++turn;
    };
    auto wait_full = [&] {
        if (!tc::mbar_wait(&full[e], turn & 1, abort)) {  // goes on without data: every barrier is still met
            if (lane == 0) set_err(p.err, MOE_ERR_TIMEOUT);
            *abort = 1;
        }
    };
    while (more(cur)) {
        const Item it = take(p, cur);
        const int rows = it.tokens * p.group;
        // this thread's two rows: what they see, and their query fragments
        int lo[2], hi[2];
        uint32_t qf[kSteps][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = rg * 16 + g + 8 * h;
            lo[h] = hi[h] = 0;
            const uint16_t* q = nullptr;
            if (r < rows) {
                const RowAt at = row_at(p, it, r);
                const int pos = it.r.kv - it.r.n + (at.token - it.r.row0);
                hi[h] = p.causal ? min(pos + 1, it.r.kv) : it.r.kv;
                lo[h] = p.window > 0 ? max(0, pos - p.window + 1) : 0;
                q = p.q + at.token * p.q_ld + at.head * p.q_head;
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                // an e4m3 row's fragments hold four neighbouring columns: k order within a step
                // is the keys' and free otherwise
                if (kFp8) {
                    const uint2 w = q ? *reinterpret_cast<const uint2*>(q + s * 16 + c * 4) : make_uint2(0, 0);
                    qf[s][h] = w.x;
                    qf[s][2 + h] = w.y;
                } else {
                    qf[s][h] = q ? *reinterpret_cast<const uint32_t*>(q + s * 16 + c * 2) : 0u;
                    qf[s][2 + h] = q ? *reinterpret_cast<const uint32_t*>(q + s * 16 + 8 + c * 2) : 0u;
                }
            }
        }
        float row_scale[2] = {p.scale_log2, p.scale_log2};
        if (kFp8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t mx = 0;  // largest magnitude as bf16 bits
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
                    mx = __vmaxu2(mx, __vmaxu2(qf[s][h] & 0x7fff7fffu, qf[s][2 + h] & 0x7fff7fffu));
                mx = max(mx & 0xffffu, mx >> 16);
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // largest element's exponent -> 14; in two factors, each a float
                const int up = 14 - ((int)(mx >> 7) - 127), u1 = up / 2, u2 = up - u1;
                row_scale[h] = p.scale_log2 * pow2(-u1) * pow2(-u2);
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        const uint32_t w = qf[s][x + h];
                        qf[s][x + h] = pack_f16x2(__uint_as_float(w << 16) * pow2(u1) * pow2(u2),
                                                  __uint_as_float(w & 0xffff0000u) * pow2(u1) * pow2(u2));
                    }
            }
        }
        uint32_t vref = 0;  // e4m3: the largest value scale byte so far
        float o[kD / 8][4];
#pragma unroll
        for (int j = 0; j < kD / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.0f, 0.0f}, base[2] = {0.0f, 0.0f};
        // keys [lo_all, hi_all) are seen by every row of the tile that sees any: no mask there
        const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile;
        const int hi_all = p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;
        const int lo_all = p.window > 0 ? max(0, pos0 + it.tokens - p.window) : 0;

        for (int kt = 0; kt < it.n; ++kt, ++tiles) {
            if (kTileGroups > 1 && (int)(tiles & 1) != tg) {
                next();
                next();
                continue;
            }
            const int ke = e;  // the ring entry of the keys; the values' is the next one
            wait_full();
            next();
            const uint32_t k_addr = tc::smem_u32(ring + ke * C::kEntryBytes);
            const uint32_t v_addr = tc::smem_u32(ring + e * C::kEntryBytes);
#pragma unroll 1
            for (int ch = 0; ch < kChunks; ++ch) {
                const int in0 = kg * kWarpKeys + ch * 16 * kStrips;  // first key within the tile
                const int key0 = (it.k0 + kt) * kKeyTile + in0;
                const bool edge = key0 < lo_all || key0 + 16 * kStrips > hi_all;
                // ---- scores
                float sc[kStrips][2][4];
#pragma unroll
                for (int st = 0; st < kStrips; ++st)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[st][0][i] = sc[st][1][i] = 0.0f;
                if (kFp8) {
#pragma unroll
                    for (int s = 0; s < kSteps; s += 2)
#pragma unroll
                        for (int st = 0; st < kStrips; ++st) {
                            uint32_t w[4];  // keys 0-7 and 8-15 of chunk s, then of chunk s + 1
                            ldsm_x4(w, k_addr + swizzled<C::kRowBytes>(
                                                    in0 + st * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), s + (lane >> 4)));
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int t = 0; t < 2; ++t) {
                                    uint32_t b0, b1;
                                    e4m3x4_f16(w[2 * u + t], b0, b1);
                                    mma16816_f16(sc[st][t], qf[s + u], b0, b1);
                                }
                        }
                } else {
#pragma unroll
                    for (int s = 0; s < kSteps; ++s)
#pragma unroll
                        for (int st = 0; st < kStrips; ++st) {
                            uint32_t b[4];
                            ldsm_x4(b, k_addr + swizzled<C::kRowBytes>(in0 + st * 16 + (lane >> 4) * 8 + (lane & 7),
                                                                       2 * s + ((lane >> 3) & 1)));
                            mma16816(sc[st][0], qf[s], b[0], b[1]);
                            mma16816(sc[st][1], qf[s], b[2], b[3]);
                        }
                }
                // ---- the keys' scales, the mask, the running maximum (before row_scale, which is > 0)
                float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
                const int mine = in0 + (lane & (16 * kStrips - 1));  // e4m3: the key whose scales this lane looks up
                const float kscale = kFp8 ? scale_of(scales[ke * kKeyTile + mine]) : 1.0f;
#pragma unroll
                for (int st = 0; st < kStrips; ++st)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        float ks[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            ks[x] = kFp8 ? __shfl_sync(0xffffffffu, kscale, st * 16 + t * 8 + c * 2 + x) : 1.0f;
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float v = sc[st][t][2 * h + x];
                                if (kFp8) v *= ks[x];
                                if (edge) {
                                    const int key = key0 + st * 16 + t * 8 + c * 2 + x;
                                    if (key < lo[h] || key >= hi[h]) v = -CUDART_INF_F;
                                }
                                sc[st][t][2 * h + x] = v;
                                mx[h] = fmaxf(mx[h], v);
                            }
                    }
                if (ch == kChunks - 1) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&empty[ke]);
                }
                if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                        const float mn = fmaxf(m[h], mx[h]);
                        const float f = m[h] == -CUDART_INF_F ? 0.0f : exp2_fast((m[h] - mn) * row_scale[h]);
                        m[h] = mn;
                        base[h] = mn == -CUDART_INF_F ? 0.0f : -mn * row_scale[h];
                        l[h] *= f;
#pragma unroll
                        for (int j = 0; j < kD / 8; ++j) {
                            o[j][2 * h] *= f;
                            o[j][2 * h + 1] *= f;
                        }
                    }
                }
                // ---- probabilities, then o += p . v
                if (ch == 0) wait_full();
                // keys of this chunk that no row sees hold anything, NaN among it: their values read as 0
                const bool tail = key0 < it.s.lo || key0 + 16 * kStrips > it.s.hi;
                float vscale = 1.0f;
                if (kFp8) {
                    const int key = key0 - in0 + mine;
                    uint32_t vb = scales[e * kKeyTile + mine];
                    if (tail && (key < it.s.lo || key >= it.s.hi)) vb = 0;
                    if (__any_sync(0xffffffffu, vb > vref)) {
                        const uint32_t to = max(vref, __reduce_max_sync(0xffffffffu, vb));
                        const float f = pow2((int)vref - (int)to);
                        vref = to;
#pragma unroll
                        for (int j = 0; j < kD / 8; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[j][i] *= f;
                    }
                    const int ex = (int)vb - (int)vref + 14 + 127;
                    vscale = vb == 255 ? CUDART_NAN_F : vb == 0 || ex <= 0 ? 0.0f : __int_as_float(ex << 23);
                }
#pragma unroll
                for (int st = 0; st < kStrips; ++st) {
                    uint32_t a[4];
                    uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of the key pairs 2c, 2c+1 and 8 further
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        float vs[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            vs[x] = kFp8 ? __shfl_sync(0xffffffffu, vscale, st * 16 + t * 8 + c * 2 + x) : 1.0f;
                        if (tail) {
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int key = key0 + st * 16 + t * 8 + c * 2 + x;
                                if (key < it.s.lo || key >= it.s.hi) keep[t] &= x ? 0x0000ffffu : 0xffff0000u;
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float p0 = exp2_fast(fmaf(sc[st][t][2 * h], row_scale[h], base[h]));
                            const float p1 = exp2_fast(fmaf(sc[st][t][2 * h + 1], row_scale[h], base[h]));
                            l[h] += p0 + p1;
                            a[2 * t + h] = kFp8 ? pack_f16x2(p0 * vs[0], p1 * vs[1]) : pack_bf16x2(p0, p1);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < C::kRowBytes * C::kHalves / 16; j += 2) {
                        uint32_t w[4];  // keys 0-7 and 8-15 of chunk j, then of chunk j + 1
                        ldsm_x4_t(w, v_addr + swizzled<C::kRowBytes>(in0 + st * 16 + ((lane >> 3) & 1) * 8 + (lane & 7),
                                                                     j + (lane >> 4)));
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if (kFp8) {
                                // bytes: a pair of keys of an even column, then of the odd one beside it
                                uint32_t w0 = __byte_perm(w[2 * u], 0, 0x3120), w1 = __byte_perm(w[2 * u + 1], 0, 0x3120);
                                if (tail) {
                                    w0 &= __byte_perm(keep[0], 0, 0x2020);
                                    w1 &= __byte_perm(keep[1], 0, 0x2020);
                                }
                                uint32_t ev0, od0, ev1, od1;
                                e4m3x4_f16(w0, ev0, od0);
                                e4m3x4_f16(w1, ev1, od1);
                                mma16816_f16(o[2 * (j + u)], a, ev0, ev1);
                                mma16816_f16(o[2 * (j + u) + 1], a, od0, od1);
                            } else {
                                if (tail) w[2 * u] &= keep[0], w[2 * u + 1] &= keep[1];
                                mma16816(o[j + u], a, w[2 * u], w[2 * u + 1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[e]);
            next();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) m[h] *= row_scale[h];  // scores in powers of two from here
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        if (kFp8) {
            const int up = (int)vref - 127 - 14, u1 = up / 2, u2 = up - u1;
#pragma unroll
            for (int j = 0; j < kD / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][i] = o[j][i] * pow2(u1) * pow2(u2);
        }
        // ---- merge the key groups: the upper half hands its state to the lower half
#pragma unroll
        for (int half = kMerged / 2; half > 0; half >>= 1) {
            float4* x = reinterpret_cast<float4*>(xchg) + ((mg % half) * kRowWarps + rg) * (kD / 8) * 32;
            float2* xm = xml + ((mg % half) * kRowWarps + rg) * 16;
            if (mg >= half && mg < 2 * half) {
#pragma unroll
                for (int j = 0; j < kD / 8; ++j) x[j * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
                if (c == 0) {
                    xm[g] = make_float2(m[0], l[0]);
                    xm[g + 8] = make_float2(m[1], l[1]);
                }
            }
            sync();
            if (mg < half) {
                float fa[2], fb[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 ml = xm[g + 8 * h];
                    const float mn = fmaxf(m[h], ml.x), b = mn == -CUDART_INF_F ? 0.0f : mn;
                    fa[h] = exp2_fast(m[h] - b);
                    fb[h] = exp2_fast(ml.x - b);
                    m[h] = mn;
                    l[h] = l[h] * fa[h] + ml.y * fb[h];
                }
#pragma unroll
                for (int j = 0; j < kD / 8; ++j) {
                    const float4 v = x[j * 32 + lane];
                    o[j][0] = o[j][0] * fa[0] + v.x * fb[0];
                    o[j][1] = o[j][1] * fa[0] + v.y * fb[0];
                    o[j][2] = o[j][2] * fa[1] + v.z * fb[1];
                    o[j][3] = o[j][3] * fa[1] + v.w * fb[1];
                }
            }
            sync();
        }
        if (mg == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = rg * 16 + g + 8 * h;
                if (r >= rows) continue;
                if (it.whole) {
                    const RowAt at = row_at(p, it, r);
                    const float inv = l[h] > 0.0f ? 1.0f / l[h] : (l[h] == 0.0f ? 0.0f : l[h]);
                    uint16_t* out = p.o + at.token * p.o_ld + at.head * p.o_head;
                    if (kFp8) {
#pragma unroll
                        for (int j = 0; j < kD / 16; ++j)
                            *reinterpret_cast<uint2*>(out + j * 16 + c * 4) =
                                make_uint2(pack_bf16x2(o[2 * j][2 * h] * inv, o[2 * j + 1][2 * h] * inv),
                                           pack_bf16x2(o[2 * j][2 * h + 1] * inv, o[2 * j + 1][2 * h + 1] * inv));
                    } else {
#pragma unroll
                        for (int j = 0; j < kD / 8; ++j)
                            *reinterpret_cast<uint32_t*>(out + j * 8 + c * 2) =
                                pack_bf16x2(o[j][2 * h] * inv, o[j][2 * h + 1] * inv);
                    }
                    if (p.lse && c == 0)
                        p.lse[(int64_t)at.token * p.heads * p.group + at.head] =
                            l[h] == 0.0f ? -CUDART_INF_F : (m[h] + log2f(l[h])) * 0.6931471805599453f;
                } else {
                    const int slot = it.first ? 0 : 1;
                    float* out = part_o(p, blockIdx.x, slot) + (size_t)r * kD;
                    if (kFp8) {
#pragma unroll
                        for (int j = 0; j < kD / 16; ++j)
                            *reinterpret_cast<float4*>(out + j * 16 + c * 4) = make_float4(
                                o[2 * j][2 * h], o[2 * j + 1][2 * h], o[2 * j][2 * h + 1], o[2 * j + 1][2 * h + 1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < kD / 8; ++j)
                            *reinterpret_cast<float2*>(out + j * 8 + c * 2) =
                                make_float2(o[j][2 * h], o[j][2 * h + 1]);
                    }
                    if (c == 0) part_ml(p, blockIdx.x, slot)[r] = make_float2(m[h], l[h]);
                }
            }
        }
        if (!it.whole)
            join<kD, kConsumers>(p, it, start.total, threadIdx.x, &last_s, sync, rows, [](int r) { return r; });
    }
}

template <int kD, bool kFp8, int kRowWarps>
cudaError_t launch_as(const moe_kv_cache& c, const Params& p, int grid, cudaStream_t st) {
    CUtensorMap km, vm;
    if (!make_pool_map(&km, c, c.k) || !make_pool_map(&vm, c, c.v)) return cudaErrorInvalidValue;
    auto kern = attn_rows_kernel<kD, kFp8, kRowWarps>;
    constexpr int smem = Cfg<kD, kFp8>::kSmem;
    cudaError_t e = ensure_max_dynamic_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, Cfg<kD, kFp8>::kThreads, smem, st, p, km, vm, c.k_scale, c.v_scale);
}

template <int kD, bool kFp8>
cudaError_t launch_rows_as(const moe_kv_cache& c, const Params& p, int row_warps, int grid, cudaStream_t st) {
    switch (row_warps) {
        case 1: return launch_as<kD, kFp8, 1>(c, p, grid, st);
        case 2: return launch_as<kD, kFp8, 2>(c, p, grid, st);
        default: return launch_as<kD, kFp8, 4>(c, p, grid, st);
    }
}

}  // namespace

cudaError_t launch_rows(const moe_kv_cache& c, Params& p, int row_warps, int grid_cap, cudaStream_t st) {
    p.tokens_per_tile = row_warps * 16 / p.group;
    const int grid = grid_for(p, grid_cap);
    const bool fp8 = c.dtype == MOE_FP8_E4M3;
    if (c.head_dim == 128)
        return fp8 ? launch_rows_as<128, true>(c, p, row_warps, grid, st)
                   : launch_rows_as<128, false>(c, p, row_warps, grid, st);
    return fp8 ? launch_rows_as<64, true>(c, p, row_warps, grid, st)
               : launch_rows_as<64, false>(c, p, row_warps, grid, st);
}

}  // namespace attn
}  // namespace moe
