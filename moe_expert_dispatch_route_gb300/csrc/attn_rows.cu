// Paged attention for query tiles of up to 64 rows (a decode step, a draft): the keys and
// values of a request are read once and HBM bounds the kernel, so the products run on
// mma.sync, whose fragments keep scores, probabilities and output in registers, and the
// warps of a CTA share out the keys of a tile instead of padding the rows to 128.
//
//   warp 8      producer: TMA copies of 128-key K and V tiles, page by page, into a ring
//   warps 0-7   row group = warp % kRowWarps (16 rows each), key group = warp / kRowWarps;
//               each keeps a running maximum and sum over its own keys; the key groups are
//               merged in shared memory once per query tile
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kConsumers = 256;
constexpr int kThreads = kConsumers + 32;
constexpr int kXchgBytes = 4 * 16 * 128 * 4;  // o of four warps

template <int kD, bool kFp8>
struct Cfg {
    static constexpr int kElt = kFp8 ? 1 : 2;
    static constexpr int kEntryBytes = kKeyTile * kD * kElt;
    static constexpr int kRowBytes = kD * kElt < 128 ? kD * kElt : 128;  // of one swizzled row
    static constexpr int kHalves = kD * kElt / kRowBytes;
    static constexpr int kEntries = kFp8 ? (kD == 128 ? 10 : 12) : (kD == 128 ? 6 : 12);
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
__global__ void __launch_bounds__(kThreads, 1)
    attn_rows_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const uint8_t* __restrict__ k_scale,
                     const uint8_t* __restrict__ v_scale) {
    using C = Cfg<kD, kFp8>;
    constexpr int kKeyWarps = 8 / kRowWarps;
    constexpr int kWarpKeys = kKeyTile / kKeyWarps;
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
            tc::mbar_init(&empty[i], 8);
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
    locate<kThreads>(p, reinterpret_cast<uint32_t*>(xchg), &start);
    Cursor cur = cursor(p, start);
    if (!more(cur)) return;

    if (warp == 8) {
        // ------------------------------------------------------------ producer
        int e = 0;
        uint32_t turn = 0;
        const int box_keys = min(p.page_size, kKeyTile), npg = kKeyTile / box_keys;
        auto next = [&] {
            if (++e == C::kEntries) e = 0, ++turn;
        };
        while (more(cur)) {
            const Item it = take(p, cur);
            const int32_t* table = p.table + (int64_t)it.b * p.table_ld;
            for (int k = 0; k < it.n; ++k) {
                const int key0 = (it.k0 + k) * kKeyTile;
                // lane i: box i of the tile (page i / kHalves of it, column half i % kHalves)
                const int pg = lane / C::kHalves, half = lane % C::kHalves;
                const int key = key0 + pg * box_keys;
                const bool want = pg < npg && key < it.s.hi && key + box_keys > it.s.lo;
                int page = 0;
                if (want) {
                    page = table[key >> p.page_shift];
                    if (page < 0 || page >= p.num_pages) {
                        set_err(p.err, MOE_ERR_BAD_INDEX);
                        page = p.num_pages;  // past the pool: the copy fills zeros
                    }
                }
                const bool scaled = kFp8 && want && half == 0 && page < p.num_pages;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, want)) * (box_keys * C::kRowBytes) +
                                       __popc(__ballot_sync(0xffffffffu, scaled)) * box_keys;
                const int off = key & (p.page_size - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
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
                    next();
                }
            }
        }
        if (*abort)  // copies still in flight land (or a bounded wait gives up) before the CTA ends
            for (int i = 0; i < C::kEntries; ++i) {
                const uint32_t issued = turn + (i < e ? 1 : 0);
                if (issued > 0) tc::mbar_wait_bounded(&full[i], (issued - 1) & 1);
            }
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int rg = warp % kRowWarps, kg = warp / kRowWarps;
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
        float o[kD / 8][4];
#pragma unroll
        for (int j = 0; j < kD / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.0f, 0.0f};
        // keys [lo_all, hi_all) are seen by every row of the tile that sees any: no mask there
        const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile;
        const int hi_all = p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;
        const int lo_all = p.window > 0 ? max(0, pos0 + it.tokens - p.window) : 0;

        for (int kt = 0; kt < it.n; ++kt) {
            const int key0 = (it.k0 + kt) * kKeyTile + kg * kWarpKeys;
            const bool edge = key0 < lo_all || key0 + kWarpKeys > hi_all;
            // ---- scores of this warp's keys
            wait_full();
            const uint32_t kt_addr = tc::smem_u32(ring + e * C::kEntryBytes);
            constexpr int kStrips = kWarpKeys / 16;
            float sc[kStrips][2][4];
#pragma unroll
            for (int st = 0; st < kStrips; ++st) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[st][0][i] = sc[st][1][i] = 0.0f;
                const int row0 = kg * kWarpKeys + st * 16;
                if (kFp8) {
#pragma unroll
                    for (int s = 0; s < kSteps; s += 2) {
                        uint32_t w[4];  // keys 0-7 and 8-15 of chunk s, then of chunk s + 1
                        ldsm_x4(w, kt_addr + swizzled<C::kRowBytes>(row0 + ((lane >> 3) & 1) * 8 + (lane & 7),
                                                                    s + (lane >> 4)));
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                uint32_t b0, b1;
                                e4m3_spread<0x1404, 0x3424>(w[2 * u + t], b0, b1);
                                mma16816(sc[st][t], qf[s + u], mul_bf16x2(b0, kTwo120), mul_bf16x2(b1, kTwo120));
                            }
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) {
                        uint32_t b[4];
                        ldsm_x4(b, kt_addr + swizzled<C::kRowBytes>(row0 + (lane >> 4) * 8 + (lane & 7),
                                                                    2 * s + ((lane >> 3) & 1)));
                        mma16816(sc[st][0], qf[s], b[0], b[1]);
                        mma16816(sc[st][1], qf[s], b[2], b[3]);
                    }
                }
            }
            // ---- scale, mask, running maximum
            float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
            for (int st = 0; st < kStrips; ++st)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int kk = st * 16 + t * 8 + c * 2 + x;
                        float f = p.scale_log2;
                        if (kFp8) f *= scale_of(scales[e * kKeyTile + kg * kWarpKeys + kk]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v = sc[st][t][2 * h + x] * f;
                            if (edge && (key0 + kk < lo[h] || key0 + kk >= hi[h])) v = -CUDART_INF_F;
                            sc[st][t][2 * h + x] = v;
                            mx[h] = fmaxf(mx[h], v);
                        }
                    }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[e]);
            next();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mn = fmaxf(m[h], mx[h]);
                    const float f = m[h] == -CUDART_INF_F ? 0.0f : exp2_fast(m[h] - mn);
                    m[h] = mn;
                    l[h] *= f;
#pragma unroll
                    for (int j = 0; j < kD / 8; ++j) {
                        o[j][2 * h] *= f;
                        o[j][2 * h + 1] *= f;
                    }
                }
            }
            // ---- probabilities (bf16 for the second product), then o += p . v
            wait_full();
            const uint32_t vt_addr = tc::smem_u32(ring + e * C::kEntryBytes);
            const float base[2] = {m[0] == -CUDART_INF_F ? 0.0f : m[0], m[1] == -CUDART_INF_F ? 0.0f : m[1]};
            // keys of this tile that no row sees hold anything, NaN among it: their values read as 0
            const bool tail = key0 < it.s.lo || key0 + kWarpKeys > it.s.hi;
#pragma unroll
            for (int st = 0; st < kStrips; ++st) {
                uint32_t a[4];
                uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of the key pairs 2c, 2c+1 and 8 further
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int kk = st * 16 + t * 8 + c * 2;
                    float vs[2] = {1.0f, 1.0f};
                    if (kFp8) {
                        vs[0] = scale_of(scales[e * kKeyTile + kg * kWarpKeys + kk]);
                        vs[1] = scale_of(scales[e * kKeyTile + kg * kWarpKeys + kk + 1]);
                    }
                    if (tail) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (key0 + kk + x < it.s.lo || key0 + kk + x >= it.s.hi) {
                                keep[t] &= x ? 0x0000ffffu : 0xffff0000u;
                                vs[x] = 0.0f;
                            }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = exp2_fast(sc[st][t][2 * h] - base[h]);
                        const float p1 = exp2_fast(sc[st][t][2 * h + 1] - base[h]);
                        l[h] += p0 + p1;
                        a[2 * t + h] = kFp8 ? pack_bf16x2(p0 * vs[0], p1 * vs[1]) : pack_bf16x2(p0, p1);
                    }
                }
                const int row0 = kg * kWarpKeys + st * 16;
#pragma unroll
                for (int j = 0; j < C::kRowBytes * C::kHalves / 16; j += 2) {
                    uint32_t w[4];  // keys 0-7 and 8-15 of chunk j, then of chunk j + 1
                    ldsm_x4_t(w, vt_addr + swizzled<C::kRowBytes>(row0 + ((lane >> 3) & 1) * 8 + (lane & 7),
                                                                  j + (lane >> 4)));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (kFp8) {
                            // 16 columns of a chunk: the even ones, then the odd ones
                            uint32_t ev0, od0, ev1, od1;
                            e4m3_spread<0x2404, 0x3414>(w[2 * u], ev0, od0);
                            e4m3_spread<0x2404, 0x3414>(w[2 * u + 1], ev1, od1);
                            if (tail) {
                                ev0 &= keep[0], od0 &= keep[0];
                                ev1 &= keep[1], od1 &= keep[1];
                            }
                            mma16816(o[2 * (j + u)], a, mul_bf16x2(ev0, kTwo120), mul_bf16x2(ev1, kTwo120));
                            mma16816(o[2 * (j + u) + 1], a, mul_bf16x2(od0, kTwo120), mul_bf16x2(od1, kTwo120));
                        } else {
                            if (tail) w[2 * u] &= keep[0], w[2 * u + 1] &= keep[1];
                            mma16816(o[j + u], a, w[2 * u], w[2 * u + 1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[e]);
            next();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        // ---- merge the key groups: the upper half hands its state to the lower half
#pragma unroll
        for (int half = kKeyWarps / 2; half > 0; half >>= 1) {
            float4* x = reinterpret_cast<float4*>(xchg) + ((kg % half) * kRowWarps + rg) * (kD / 8) * 32;
            float2* xm = xml + ((kg % half) * kRowWarps + rg) * 16;
            if (kg >= half && kg < 2 * half) {
#pragma unroll
                for (int j = 0; j < kD / 8; ++j) x[j * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
                if (c == 0) {
                    xm[g] = make_float2(m[0], l[0]);
                    xm[g + 8] = make_float2(m[1], l[1]);
                }
            }
            sync();
            if (kg < half) {
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
        if (kg == 0) {
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
    return launch_pdl(kern, grid, kThreads, smem, st, p, km, vm, c.k_scale, c.v_scale);
}

template <int kD, bool kFp8>
cudaError_t launch_rows_as(const moe_kv_cache& c, const Params& p, int row_warps, int grid, cudaStream_t st) {
    switch (row_warps) {
        case 1: return launch_as<kD, kFp8, 1>(c, p, grid, st);
        case 2: return launch_as<kD, kFp8, 2>(c, p, grid, st);
        case 4: return launch_as<kD, kFp8, 4>(c, p, grid, st);
        default: return launch_as<kD, kFp8, 8>(c, p, grid, st);
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
