// Paged attention for query tiles of up to 256 rows (prompt chunks): bound by the tensor cores,
// so both products run on tcgen05 with scores, probabilities and output in tensor memory.
//
// A query tile is two halves of up to 128 rows over the same key tiles; while the softmax of
// one half runs, the tensor cores work on the other.  Per half and 128-key tile:
//   S = Q K^T    A = Q (shared memory), B = K tile (d contiguous), 128 columns of fp32
//   P = 2^(s - m) in 16 bits, written over S's first 64 columns: the A operand of
//   O += P V     A = P (tensor memory), B = V tile with the columns contiguous
// which fills the 512 columns of tensor memory: S0 | S1 | O0 | O1.  The MMA thread issues
// PV(j), S(j+1) for each half in turn; tcgen05.mma instructions of one thread execute in
// order, so S(j+1) may overwrite P(j) without a wait.
//
// What bounds it: the chain of one half's scores, softmax and product, which two halves in turn cover
// in part; a pair of tiles (both halves, 128 keys, head_dim 128) takes 3400 cycles.  Its 32 MMAs
// last 2070 (64.7 each), during which they read 192 KB of operands and the copies write 64 KB at
// 128 bytes a cycle, 2048: shared memory is as busy as the tensor cores, which stretches them to
// 2450.  8192 rows over 16384 tokens, 32 / 4 heads of 128, bf16: 1100-1165 us from box to box, 1420-1500
// TFLOP/s (64 columns: 974 us for half the products; the softmax is the same).
//
// The running maximum is followed loosely: o and the sum stay relative to an older maximum
// until a row's new one is 2^8 times as large (in the probabilities), and only then are they
// rescaled.  The quotient o / sum does not depend on the reference point, fp32 holds both
// with the same relative precision, and bf16 probabilities up to 256 round like those up to 1.
// So the rescaling, a round trip of o through registers, happens a few times a row.
//
// An e4m3 cache is multiplied in fp16: a conversion instruction and a product turn two codes
// into two elements (bf16 takes ten for four: shifts, masks and products).  What is multiplied is
//   q   a row times a power of two that brings its largest element into [2^14, 2^15); what lies
//       2^29 below that is off by 2^-40 of the largest
//   k   code * 2^(s - r), s the key's scale exponent, r a reference at most 2^15 above it: exact
//   v   likewise, with a reference to which o refers and that is at most 2^12 above (attn.cuh)
//   p   2^7 p
// A tile whose scales lie elsewhere holds the codes as they are: its scores are multiplied by 2^s and its part
// of o is added up in fp32 by the softmax's threads, several times as long.
// The same chunk takes 1456 us: the conversion shares shared memory and issue slots with the rest
// (left out, when this took 1540, it left 1250).
//
//   warps 0-3, 4-7   softmax and epilogue of half 0, 1 (a thread owns a row; e4m3: its row of Q too)
//   warps 8-11       e4m3 only: turn raw K and V tiles into fp16 tiles
//   last four warps  one issues the MMAs, one the copies
#include <cudaTypedefs.h>

#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kHalfRows = 128;
// Tiles whose references and scales are kept.  The warps that come to tile t have had the ring's entry that the
// values of tile t - 3 held (of 6 entries: t - 4), so those of at most four tiles are in use.
constexpr int kRefs = 4;
constexpr int kSpread = 15;  // fp16 holds an e4m3 code times 2^-15 exactly

template <int kD, bool kFp8>
struct Cfg {
    static constexpr int kThreads = kFp8 ? 512 : 384;
    static constexpr int kCols = kD / 64;                             // 128-byte column blocks of a 16-bit tile
    static constexpr int kBlockBytes = kKeyTile * 128;                // one of them
    static constexpr int kQBytes = 2 * kCols * kHalfRows * 128;       // both halves of Q
    static constexpr int kEntryBytes = kCols * kBlockBytes;           // a K or V tile of 16-bit elements
    static constexpr int kRawBytes = kKeyTile * kD;                   // an e4m3 one
    static constexpr int kEntries = kFp8 ? (kD == 64 ? 6 : 4) : kD == 64 ? 8 : 5;
    static constexpr int kRaw = kFp8 ? (kD == 64 ? 6 : 2) : 0;
    // e4m3: raw tiles, their scales; of kRefs tiles the keys' and values' scales and references
    static constexpr int kFp8Bytes = kFp8 ? kRaw * (kRawBytes + kKeyTile) + kRefs * (2 * kKeyTile + 4) : 0;
    static constexpr int kBars = 2 * (kEntries + kRaw) + 2 + 6 + 1 + kRefs + 2;  // 8 bytes each
    static constexpr int kTail = (8 * kBars + 4 * (kEntries + kRaw) + 15) / 16 * 16;
    static constexpr int kSmem = 1024 + kQBytes + kEntries * kEntryBytes + kFp8Bytes + kTail;
    static_assert(kSmem <= 232448 - 256, "");
    static_assert(kEntries * kEntryBytes >= (kMaxRequests + 32) * 4, "locate()'s scratch");
    // registers per thread after the redistribution: softmax, converters, the rest; their sum
    // over the block is what it was launched with
    static constexpr int kRegsSoft = kFp8 ? 168 : 192;
    static constexpr int kRegsConv = 80;
    static constexpr int kRegsRest = kFp8 ? 96 : 120;
};

// ---------------------------------------------------------------- PTX not shared with the FFN
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem], A's row i in lane i, two 16-bit elements of K per column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an operand whose M/N index is contiguous (here V: columns contiguous, keys the
// K index), 128-byte swizzle: blocks of 64 columns kBlock bytes apart (the leading byte
// offset), groups of 8 keys 1024 bytes apart (the stride byte offset).
__device__ __forceinline__ uint64_t desc_sw128_mnmajor(uint32_t saddr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(block_bytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
constexpr uint32_t kIdescBMn = 1u << 16;  // B with its N index contiguous

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
          "l"(*reinterpret_cast<uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The halves of a query tile: rows, and the key tiles each sees within an item's.
struct Halves {
    int rows;     // rows of a full half: tokens_per_tile / 2 * group
    int count;    // 1 or 2
    int k0[2], k1[2];
};
__device__ __forceinline__ Halves halves(const Params& p, const Item& it) {
    Halves v;
    const int half = p.tokens_per_tile / 2;
    v.rows = half * p.group;
    v.count = it.tokens > half ? 2 : 1;
    const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t0 = h * half, t1 = min(t0 + half, it.tokens);
        const int hi = p.causal ? min(it.r.kv, max(pos0 + t1, 0)) : it.r.kv;
        const int lo = p.window > 0 ? max(0, pos0 + t0 - p.window + 1) : 0;
        v.k0[h] = max(lo / kKeyTile, it.k0);
        v.k1[h] = h < v.count && hi > lo ? min((hi + kKeyTile - 1) / kKeyTile, it.k0 + it.n) : 0;
    }
    return v;
}
__device__ __forceinline__ bool active(const Halves& v, int h, int kt) { return kt >= v.k0[h] && kt < v.k1[h]; }

// What the MMA warp has to know of a K or V tile, put beside it by the copying warp: so it keeps
// no account of query tiles itself, and its registers go to descriptors.  (With the account in
// it, the spilled descriptors cost more than the MMAs: 110 cycles an instruction instead of 65.)
enum : uint32_t {
    kAct0 = 1u,       // half 0 (1: half 1) uses this tile; for V,
    kFirst0 = 4u,     // it is the first one of half 0 (1)
    kNewQ = 16u,      // K: the first tile of a query tile
    kLastK = 32u,     // K: the last one
    kStop = 64u,      // no more tiles
    kSeenLo = 8,      // bits 8-15: first key of the tile that any row sees, 16-23: one past the last
    kSeenHi = 16
};

// One thread: the sum of row r of n parts of a split tile, those of CTAs first, first + step, ..., in
// this order.  kLast: it goes to the output, otherwise to the place of the first part.
constexpr int kFan = 4;  // the most parts summed together
template <int kD, bool kLast>
__device__ void join_row(const Params& p, const Parts& parts, int first, int step, int n, const RowAt& at, int r) {
    auto ml_of = [&](int i) {
        const int c = first + i * step;
        return __ldcg(part_ml(p, c, part_slot(parts, c)) + r);
    };
    float2 ml[kFan];
    float m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
    for (int i = 0; i < kFan; ++i) ml[i] = i < n ? ml_of(i) : make_float2(-CUDART_INF_F, 0.0f);
#pragma unroll
    for (int i = 0; i < kFan; ++i) m = fmaxf(m, ml[i].x);
    const float to = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < kFan; ++i) l += ml[i].y * exp2_fast(ml[i].x - to);
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    uint16_t* out = p.o + at.token * p.o_ld + at.head * p.o_head;
    float4* sum = reinterpret_cast<float4*>(part_o(p, first, part_slot(parts, first))) + r;
    // batches of columns one after another, each over all parts, in one rolled loop: this code is cold in
    // the instruction caches; the next loads go out before a batch is stored
    constexpr int kBatch = 8;  // loads under way together, four columns each
    float4 x[kBatch], o[kBatch];
    float f;
    int load_b = 0, load_i = 0;
    auto load = [&] {
        if (load_b >= kD / 4) return;
        const int c = first + load_i * step;
        const float4* from = reinterpret_cast<const float4*>(part_o(p, c, part_slot(parts, c))) + r;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) x[j] = __ldcg(from + (load_b + j) * kMaxRows);
        f = ml_of(load_i).x;
        if (++load_i == n) load_i = 0, load_b += kBatch;
    };
    auto clear = [&] {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    };
    clear();
    load();
    int i = 0;
#pragma unroll 1
    for (int b = 0; b < kD / 4;) {
        const float w = exp2_fast(f - to);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            o[j].x += x[j].x * w, o[j].y += x[j].y * w;
            o[j].z += x[j].z * w, o[j].w += x[j].w * w;
        }
        load();
        if (++i < n) continue;
        if (kLast) {
#pragma unroll
            for (int j = 0; j < kBatch; j += 2)
                *reinterpret_cast<uint4*>(out + (b + j) * 4) = make_uint4(
                    cvt_bf16x2(o[j].x * inv, o[j].y * inv), cvt_bf16x2(o[j].z * inv, o[j].w * inv),
                    cvt_bf16x2(o[j + 1].x * inv, o[j + 1].y * inv), cvt_bf16x2(o[j + 1].z * inv, o[j + 1].w * inv));
        } else {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) sum[(b + j) * kMaxRows] = o[j];
        }
        clear();
        i = 0;
        b += kBatch;
    }
    if (!kLast)
        part_ml(p, first, part_slot(parts, first))[r] = make_float2(m, l);
    else if (p.lse)
        p.lse[(int64_t)at.token * p.heads * p.group + at.head] =
            l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
}

// The softmax threads of a CTA whose part of a split tile is stored; r and `at` are the thread's row,
// if valid.  A part is up to 128 KB, which a CTA takes two microseconds to add, so parts are
// summed kFan at a time, each group by the last of its CTAs to arrive, and the sums again: one
// request's 256 rows a head over 16384 tokens, 38 parts a tile: 42 us, 95 with one CTA adding them
// all; groups of 6 or 8 take 6 us more than groups of 4.  The counter is that of a group's second
// member, which is the second of no other group.
template <int kD, typename Sync>
__device__ void join(const Params& p, const Item& it, const Start& st, const RowAt& at, int r, bool valid, int* flag,
                     Sync sync) {
    const Parts parts = parts_of(p, it, st);
    const int n = parts.last - parts.first + 1;
    int step = 1;
    if (n > kFan) {
        const int me = (int)blockIdx.x - parts.first;
        for (; step * kFan < n; step *= kFan) {
            const int head = me / (step * kFan) * (step * kFan), members = min(kFan, (n - head + step - 1) / step);
            if (members == 1) continue;
            const int first = parts.first + head;
            if (!last_of(p.counters + first + step, members, threadIdx.x, flag, sync)) return;
            if (valid) join_row<kD, false>(p, parts, first, step, members, at, r);
        }
    }
    const int members = (n + step - 1) / step;
    if (last_of(p.counters + parts.first + step, members, threadIdx.x, flag, sync) && valid)
        join_row<kD, true>(p, parts, parts.first, step, members, at, r);
}

// One thread: counts the parts of a CTA that gives up, as if they had been stored.
template <int kD>
__device__ __noinline__ void let_go(const Params& p, const Start& st, int* flag) {
    for (Cursor cur = cursor(st); more(cur);) {
        const Item it = take(p, cur);
        if (!it.whole) join<kD>(p, it, st, RowAt{0, 0}, 0, false, flag, [] {});
    }
}

template <int kD, bool kFp8>
__global__ void __launch_bounds__(Cfg<kD, kFp8>::kThreads, 1)
    attn_tile_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const uint8_t* __restrict__ k_scale, const uint8_t* __restrict__ v_scale) {
    using C = Cfg<kD, kFp8>;
    extern __shared__ uint8_t smem_raw[];
    // aligned by an offset: rounding the address itself would make every access a generic one, with
    // 64-bit addresses (e4m3 1560 us instead of 1445, bf16 1145 instead of 1123)
    uint8_t* qs = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);
    uint8_t* ring = qs + C::kQBytes;                          // bf16 tiles, as the MMAs read them
    uint8_t* raw = ring + C::kEntries * C::kEntryBytes;       // e4m3 tiles
    uint8_t* scales = raw + C::kRaw * C::kRawBytes;
    // e4m3, of the last kRefs tiles: scale bytes of keys and values; references of both, bit 16: far apart
    uint8_t* tile_scales = scales + C::kRaw * kKeyTile;
    uint32_t* tile_refs = reinterpret_cast<uint32_t*>(tile_scales + kRefs * 2 * kKeyTile);
    uint64_t* full = reinterpret_cast<uint64_t*>(raw + C::kFp8Bytes);
    uint64_t* empty = full + C::kEntries;
    uint64_t* raw_full = empty + C::kEntries;
    uint64_t* raw_empty = raw_full + C::kRaw;
    uint64_t* q_full = raw_empty + C::kRaw;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;   // [2] scores of a half are in tensor memory
    uint64_t* p_full = s_full + 2;    // [2] its probabilities are
    uint64_t* pv_done = p_full + 2;   // [2] they have been multiplied into o
    uint64_t* q_ready = pv_done + 2;  // e4m3: Q has been turned into fp16
    uint64_t* ref_full = q_ready + 1;  // e4m3, [kRefs]: a V tile's reference is there
    uint64_t* done = ref_full + kRefs;
    uint64_t* never = done + 1;
    uint32_t* cmds = reinterpret_cast<uint32_t*>(never + 1);  // of the ring's tiles, then of the raw ones
    uint32_t* raw_cmds = cmds + C::kEntries;
    __shared__ Start start;
    __shared__ Cursor cursors[2];  // where the two softmax groups stand: not held in registers
    __shared__ int abort_s, last_s;
    __shared__ uint32_t tmem_s;
    volatile int* abort = &abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMmaWarp = C::kThreads / 32 - 4, kCopyWarp = kMmaWarp + 1;
    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int i = 0; i < C::kEntries; ++i) {
            tc::mbar_init(&full[i], kFp8 ? 4 : 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kRaw; ++i) {
            tc::mbar_init(&raw_full[i], 1);
            tc::mbar_init(&raw_empty[i], 4);
        }
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_empty, 1);
        for (int h = 0; h < 2; ++h) {
            tc::mbar_init(&s_full[h], 1);
            tc::mbar_init(&p_full[h], 4);
            tc::mbar_init(&pv_done[h], 1);
        }
        tc::mbar_init(q_ready, 8);
        for (int i = 0; i < kRefs; ++i) tc::mbar_init(&ref_full[i], 1);
        tc::mbar_init(done, 1);
        tc::mbar_init(never, 1);
        tc::fence_barrier_init();
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&vmap);
    }
    __syncthreads();
    pdl_begin();
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_s, 512);
        tc::tmem_relinquish();
        tc::tc_fence_before();
    }
    locate<C::kThreads>(p, reinterpret_cast<uint32_t*>(ring), &start);
    tc::tc_fence_after();
    const uint32_t tmem = tmem_s;
    if (p.inject_ns > 0 && blockIdx.x == 0) {  // test hook: the failure path of a bounded wait
        if (threadIdx.x == 0) {
            tc::wait_on_nothing(never, (uint64_t)p.inject_ns);
            set_err(p.err, MOE_ERR_TIMEOUT);
            let_go<kD>(p, start, &last_s);
        }
        __syncthreads();
        if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
        return;
    }
    Cursor cur = cursor(start);
    if (threadIdx.x == 0 || threadIdx.x == 128) cursors[threadIdx.x >> 7] = cur;
    __syncthreads();
    // a wait that runs out is reported and then passed, here and in every later wait, so that
    // each barrier is still met; the results are void
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!tc::mbar_wait(bar, parity, abort)) {
            set_err(p.err, MOE_ERR_TIMEOUT);
            *abort = 1;
        }
    };

    if (warp >= kMmaWarp) {
        regs_dec<C::kRegsRest>();
        if (warp == kCopyWarp) {
            // -------------------------------------------------------- copies
            int e = 0;
            uint32_t turn = 0, items = 0, sent = 0, q_sent = 0;
            const int box_keys = min(p.page_size, kKeyTile), npg = kKeyTile / box_keys;
            constexpr int kBoxes = kFp8 ? 1 : C::kCols;  // column blocks of a K or V tile as copied
            constexpr int kRing = kFp8 ? C::kRaw : C::kEntries;
            constexpr int kRowBytes = kFp8 ? kD : 128;
            uint64_t* to_full = kFp8 ? raw_full : full;
            uint64_t* to_empty = kFp8 ? raw_empty : empty;
            const int half_tokens = p.tokens_per_tile / 2;
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
                if (it.n == 0) {
                    ahead();
                    continue;
                }
                const Halves v = halves(p, it);
                if (items > 0) wait(q_empty, (items - 1) & 1);
                const bool go = !*abort;
                if (go) ++q_sent;
                if (go && lane == 0) {
                    const int count = it.tokens > half_tokens ? 2 : 1;
                    tc::mbar_arrive_expect_tx(q_full, count * C::kCols * half_tokens * p.group * 128);
                    for (int h = 0; h < count; ++h)
                        for (int b = 0; b < C::kCols; ++b)
                            tc::tma_load_3d(qs + (h * C::kCols + b) * kHalfRows * 128, &qmap, q_full, b * 64,
                                            it.head * p.group,
                                            it.r.row0 + it.tile * p.tokens_per_tile + h * half_tokens);
                }
                ++items;
                for (int k = 0; k < it.n; ++k) {
                    const int key0 = (it.k0 + k) * kKeyTile;
                    // lane i: box i of the tile (page i / kBoxes of it, column block i % kBoxes)
                    const int pg = lane / kBoxes, blk = lane % kBoxes;
                    const int key = key0 + pg * box_keys;
                    const bool want = pg < npg && key < it.s.hi && key + box_keys > it.s.lo;
                    int page = page_of(p, it, pages, key0, pg);
                    if (want && (page < 0 || page >= p.num_pages)) {
                        set_err(p.err, MOE_ERR_BAD_INDEX);
                        page = p.num_pages;  // past the pool: the copy fills zeros
                    }
                    const bool scaled = kFp8 && want && page < p.num_pages;
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, want)) * (box_keys * kRowBytes) +
                                           __popc(__ballot_sync(0xffffffffu, scaled)) * box_keys;
                    const int off = key & (p.page_size - 1), kt = it.k0 + k;
                    uint32_t cmd = (uint32_t)min(max(it.s.lo - key0, 0), kKeyTile) << kSeenLo |
                                   (uint32_t)min(it.s.hi - key0, kKeyTile) << kSeenHi;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (active(v, h, kt)) cmd |= kAct0 << h | (kt == v.k0[h] ? kFirst0 << h : 0);
                    if (k == 0) cmd |= kNewQ;
                    if (k == it.n - 1) cmd |= kLastK;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        if (turn > 0) wait(&to_empty[e], (turn - 1) & 1);
                        if (lane == 0) (kFp8 ? raw_cmds : cmds)[e] = cmd;
                        if (kFp8 && want && !scaled)  // a page outside the pool: its tokens read as zeros
                            for (int i = 0; i < box_keys; ++i) scales[e * kKeyTile + pg * box_keys + i] = 0;
                        if (!*abort) {
                            ++sent;
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive_expect_tx(&to_full[e], bytes);
                            __syncwarp();
                            uint8_t* dst = kFp8 ? raw + e * C::kRawBytes + pg * box_keys * kD
                                                : ring + e * C::kEntryBytes + blk * C::kBlockBytes + pg * box_keys * 128;
                            if (want)
                                tc::tma_load_4d(dst, kv ? &vmap : &kmap, &to_full[e], blk * 64, off, it.head, page);
                            if (scaled)
                                tc::bulk_load(scales + e * kKeyTile + pg * box_keys,
                                              (kv ? v_scale : k_scale) +
                                                  ((int64_t)page * p.heads + it.head) * p.page_size + off,
                                              box_keys, &to_full[e]);
                        }
                        if (++e == kRing) e = 0, ++turn;
                    }
                    if (k == 0) ahead();
                }
            }
            if (*abort) {  // copies still in flight land (or a bounded wait gives up) before the CTA ends
                for (int i = 0; i < kRing; ++i) {
                    const uint32_t times = (sent + kRing - 1 - i) / kRing;  // that entry i has been copied to
                    if (times > 0) tc::mbar_wait_bounded(&to_full[i], (times - 1) & 1);
                }
                if (q_sent > 0) tc::mbar_wait_bounded(q_full, (q_sent - 1) & 1);
            }
            if (turn > 0) wait(&to_empty[e], (turn - 1) & 1);
            if (lane == 0) {
                (kFp8 ? raw_cmds : cmds)[e] = kStop;
                tc::mbar_arrive(&to_full[e]);
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------- MMAs
            // operand formats: 1 bf16, 0 fp16
            constexpr uint32_t kFormat = kFp8 ? tc::idesc_bf16_f32(0, 0) & ~(1u << 4) : 0;
            constexpr uint32_t kIdescS = tc::idesc_bf16_f32(128, kKeyTile) & ~kFormat;
            constexpr uint32_t kIdescO = (tc::idesc_bf16_f32(128, kD) | kIdescBMn) & ~kFormat;
            int e = 0;
            uint32_t turn = 0, queries = 0;
            uint32_t np0 = 0, np1 = 0;  // probabilities of a half taken so far
            const uint64_t q_desc = tc::desc_sw128_kmajor(tc::smem_u32(qs));
            const uint64_t k_desc = tc::desc_sw128_kmajor(tc::smem_u32(ring));
            const uint64_t v_desc = desc_sw128_mnmajor(tc::smem_u32(ring), C::kBlockBytes);
            auto next = [&] {
                if (++e == C::kEntries) e = 0, ++turn;
            };
            auto scores = [&](int h, int at) {  // S_h = Q_h K^T from ring entry `at`
                if (tc::elect_one()) {
                    // a step along K moves a descriptor's start address, its low bits (in 16 bytes)
                    const uint64_t a = q_desc + (uint32_t)(h * (C::kCols * kHalfRows * 128 >> 4));
                    const uint64_t b = k_desc + (uint32_t)(at * (C::kEntryBytes >> 4));
#pragma unroll
                    for (int s = 0; s < kD / 16; ++s) {
                        const uint32_t off = ((s / 4) * C::kBlockBytes + (s % 4) * 32) >> 4;
                        tc::mma_bf16(tmem + h * 128, a + off, b + off, kIdescS, s > 0);
                    }
                    tc::mma_commit(&s_full[h]);
                }
                __syncwarp();
            };
            auto values = [&](int h, int at, uint32_t accumulate) {  // O_h (+)= P_h V
                if (tc::elect_one()) {
                    const uint64_t b = v_desc + (uint32_t)(at * (C::kEntryBytes >> 4));
#pragma unroll
                    for (int s = 0; s < kKeyTile / 16; ++s)
                        mma_bf16_ta(tmem + 256 + h * 128, tmem + h * 128 + s * 8, b + s * (2048 >> 4), kIdescO,
                                    s > 0 ? 1u : accumulate);
                    tc::mma_commit(&pv_done[h]);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* bar) {
                if (tc::elect_one()) tc::mma_commit(bar);
                __syncwarp();
            };
            // K tile at e is there: its command, with Q there too
            auto keys = [&]() -> uint32_t {
                wait(&full[e], turn & 1);
                const uint32_t cmd = cmds[e];
                if (cmd & kNewQ) wait(kFp8 ? q_ready : q_full, queries++ & 1);
                tc::tc_fence_after();
                return cmd;
            };
            auto keys_done = [&](uint32_t cmd) {
                commit(&empty[e]);
                if (cmd & kLastK) commit(q_empty);
                next();
            };
            uint32_t cmd = keys();
            if (!(cmd & kStop)) {
                if (cmd & kAct0) scores(0, e);
                if (cmd & (kAct0 << 1)) scores(1, e);
                keys_done(cmd);
            }
            while (!(cmd & kStop)) {
                const int ve = e;
                wait(&full[ve], turn & 1);
                const int z0 = cmd >> kSeenLo & 255, z1 = cmd >> kSeenHi & 255;
                if (!kFp8 && (z0 > 0 || z1 < kKeyTile)) {
                    // keys that no row sees hold anything, NaN among it: 0 * NaN would reach o
                    uint4* row = reinterpret_cast<uint4*>(ring + ve * C::kEntryBytes);
                    for (int i = lane; i < kKeyTile * 8; i += 32)
                        if (i / 8 < z0 || i / 8 >= z1)
#pragma unroll
                            for (int b = 0; b < C::kCols; ++b)
                                row[b * (C::kBlockBytes / 16) + i] = make_uint4(0, 0, 0, 0);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                next();
                // within a query tile the next scores of a half follow its product at once; those of
                // another query tile wait for its rows, and both halves' products come first
                const bool last = cmd & kLastK;
                uint32_t then = 0;
                if (cmd & kAct0) {
                    wait(&p_full[0], np0++ & 1);
                    tc::tc_fence_after();
                    values(0, ve, cmd & kFirst0 ? 0 : 1);
                }
                if (!last) {
                    then = keys();
                    if (then & kAct0) scores(0, e);
                }
                if (cmd & (kAct0 << 1)) {
                    wait(&p_full[1], np1++ & 1);
                    tc::tc_fence_after();
                    values(1, ve, cmd & (kFirst0 << 1) ? 0 : 1);
                }
                commit(&empty[ve]);
                if (last) {
                    then = keys();
                    if (then & kAct0) scores(0, e);
                }
                if (then & (kAct0 << 1)) scores(1, e);
                if (!(then & kStop)) keys_done(then);
                cmd = then;
            }
            commit(done);
            tc::mbar_wait_bounded(done, 0);
        }
    } else if (kFp8 && warp >= 8) {
        // ------------------------------------------------------------ e4m3 tiles to fp16
        regs_dec<C::kRegsConv>();
        int re = 0, e = 0;
        uint32_t rturn = 0, turn = 0, tile = 0;
        int k_ref = 1;  // of the last tile of keys
        bool k_far = false;
        Scales vs = {0, 8, 0, 0};  // of the query tile's values
        // A warp turns 32 keys, 8 at a time.  Eight lanes read four chunks of rows r and r ^ 5:
        // under the 128-byte swizzle both the 16-byte reads and the two 16-byte writes of each
        // lane fall into different banks.
        const int quad = lane >> 2, c4 = lane & 3;
        const int row8 = (quad >> 1) ^ ((quad & 1) * 5);
        for (uint32_t i = 0;; ++i) {  // K, V, K, V, ...
            wait(&raw_full[re], rturn & 1);
            const uint32_t cmd = raw_cmds[re];
            const bool values = i & 1;
            const int z0 = cmd >> kSeenLo & 255, z1 = cmd >> kSeenHi & 255;
            const uint8_t* sc = scales + re * kKeyTile;
            // the reference of the tile's scales, and whether they are too far from it
            const bool edge = z0 > 0 || z1 < kKeyTile;
            if (values && (cmd & kNewQ)) vs = {0, 8, 0, 0};
            int ref = values ? (int)vs.ref : k_ref;
            bool far = values && k_far;
            if (!(cmd & kStop)) {
                uint32_t four = reinterpret_cast<const uint32_t*>(sc)[lane];
                if (edge) {  // 255 for keys that are not seen: like NaN, it counts for nothing
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (lane * 4 + j < z0 || lane * 4 + j >= z1) four |= 255u << (8 * j);
                }
                // the largest byte + 1, 255 wrapping to 0, and the smallest, two bytes at a time
                const uint32_t even = four & 0xff00ffu, odd = four >> 8 & 0xff00ffu;
                const uint32_t mx2 = __vmaxu2((even + 0x10001u) & 0xff00ffu, (odd + 0x10001u) & 0xff00ffu);
                const uint32_t mn2 = __vminu2(even, odd), mx = max(mx2 & 255, mx2 >> 16), mn = min(mn2 & 255, mn2 >> 16);
                if (__any_sync(0xffffffffu, (int)mx > ref + 1 || (int)mn < ref - (values ? (int)vs.span : kSpread))) {
                    const int top = (int)__reduce_max_sync(0xffffffffu, mx) - 1;
                    const int low = __reduce_min_sync(0xffffffffu, mn);
                    if (!values) {
                        k_ref = ref = max(top, 1);  // 2^(ref - 127) is a normal number
                        far = top - low > kSpread;
                    } else {
                        take_in(vs, low, top);
                        // 2^(ref - 127 - kPBits), the unit of o, is a normal number
                        vs.ref = max(vs.ref, 8u);
                        ref = vs.ref;
                        far |= !near_ref(vs, low, top);
                    }
                }
                if (!values) k_far = far;
                if (warp == 8) {  // for the softmax
                    const uint32_t known = values || far ? four : ref * 0x01010101u;
                    reinterpret_cast<uint32_t*>(tile_scales)[(tile % kRefs * 2 + values) * 32 + lane] = known;
                    __syncwarp();
                    if (values && lane == 0) {
                        tile_refs[tile % kRefs] = k_ref | ref << 8 | (far ? 1u << 16 : 0u);
                        tc::mbar_arrive(&ref_full[tile % kRefs]);
                    }
                }
            }
            if (turn > 0) wait(&empty[e], (turn - 1) & 1);
            if (lane == 0 && warp == 8) cmds[e] = cmd;
            if (cmd & kStop) {
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&full[e]);
                break;
            }
            if (values) ++tile;
            const uint8_t* src = raw + re * C::kRawBytes;
            uint8_t* dst = ring + e * C::kEntryBytes;
            auto chunk_at = [&](int r, int hf) {
                return *reinterpret_cast<const uint4*>(src + (kD == 128 ? r * 128 + (((hf * 4 + c4) ^ (r & 7)) << 4)
                                                                        : r * 64 + ((c4 ^ ((r >> 1) & 3)) << 4)));
            };
            // lane i: the factor of key 32 * (warp - 8) + i: 2^ex in fp16, subnormal below 2^-14
            uint32_t factor;
            {
                const int key = (warp - 8) * 32 + lane, b = sc[key];
                const int ex = far ? 0 : b - ref;  // far: the codes as they are
                factor = (b == 255    ? 0x7e00u
                          : ex >= -14 ? (uint32_t)(ex + 15) << 10
                          : ex >= -24 ? 1u << (ex + 24)
                                      : 0u) *
                         0x10001u;
                if (key < z0 || key >= z1) factor = 0;
            }
            const int first = (warp - 8) * 32 + row8;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                const int r = first + g * 8;
                uint4 w[C::kCols];
#pragma unroll
                for (int hf = 0; hf < C::kCols; ++hf) w[hf] = chunk_at(r, hf);
                const uint32_t f = __shfl_sync(0xffffffffu, factor, g * 8 + row8);
                if (edge && (r < z0 || r >= z1)) {
#pragma unroll
                    for (int hf = 0; hf < C::kCols; ++hf) w[hf] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int hf = 0; hf < C::kCols; ++hf) {
                    const uint32_t x[4] = {w[hf].x, w[hf].y, w[hf].z, w[hf].w};
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e4m3x4_f16(x[j], o[2 * j], o[2 * j + 1]);
                        o[2 * j] = mul_f16x2(o[2 * j], f);
                        o[2 * j + 1] = mul_f16x2(o[2 * j + 1], f);
                    }
                    uint8_t* to = dst + hf * C::kBlockBytes + r * 128;
                    *reinterpret_cast<uint4*>(to + (((2 * c4) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(to + (((2 * c4 + 1) ^ (r & 7)) << 4)) =
                        make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&full[e]);
                tc::mbar_arrive(&raw_empty[re]);
            }
            if (++re == C::kRaw) re = 0, ++rturn;
            if (++e == C::kEntries) e = 0, ++turn;
        }
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        regs_inc<C::kRegsSoft>();
        const int h = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter of the lanes
        const uint32_t ts = tmem + h * 128 + lanes, to = tmem + 256 + h * 128 + lanes;
        auto sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        uint32_t n = 0;  // key tiles of this half so far
        uint32_t tiles = 0, queries = 0;  // key tiles, and query tiles with any, of both halves
        for (;;) {
            Cursor c = cursors[h];
            if (!more(c)) break;
            Item it = take(p, c);
            Halves v = halves(p, it);
            const int q = h * v.rows + row;  // row of the query tile
            const bool valid = row < v.rows && q < it.tokens * p.group;
            int lo = 0, hi = 0;
            RowAt at = {0, 0};
            if (valid) {
                at = row_at(p, it, q);
                const int pos = it.r.kv - it.r.n + (at.token - it.r.row0);
                hi = p.causal ? min(pos + 1, it.r.kv) : it.r.kv;
                lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
            }
            // every row of the half sees keys [lo_all, hi_all): no mask there
            const int half = p.tokens_per_tile / 2;
            const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile + h * half;
            const int pos1 = pos0 + min(half, it.tokens - h * half) - 1;
            const int hi_all = p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;
            const int lo_all = p.window > 0 ? max(0, pos1 - p.window + 1) : 0;
            float m = -CUDART_INF_F, l = 0.0f;  // m in powers of two
            float row_scale = p.scale_log2;
            int o_ref = 127 + kPBits;  // e4m3: o is in units of 2^(o_ref - 127 - kPBits)
            if (kFp8 && it.n > 0) {
                // this thread's row of Q into fp16, in place
                wait(q_full, queries++ & 1);
                if (h < v.count) {
                    uint8_t* q_row = qs + h * C::kCols * kHalfRows * 128 + row * 128;
                    uint32_t mx = 0;  // largest magnitude as bf16 bits
#pragma unroll 4
                    for (int c = 0; c < kD / 8; ++c) {
                        const uint4 x = *reinterpret_cast<const uint4*>(q_row + (c >> 3) * kHalfRows * 128 +
                                                                        (((c & 7) ^ (row & 7)) << 4));
                        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
                    }
                    const int up = f16_row_exp(max(mx & 0xffffu, mx >> 16)), u1 = up / 2;
                    const float f1 = pow2(u1), f2 = pow2(up - u1);
                    row_scale = p.scale_log2 * pow2(-u1) * pow2(u1 - up);
#pragma unroll 4
                    for (int c = 0; c < kD / 8; ++c) {
                        uint4* at = reinterpret_cast<uint4*>(q_row + (c >> 3) * kHalfRows * 128 +
                                                             (((c & 7) ^ (row & 7)) << 4));
                        const uint4 x = *at;
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                        uint32_t f[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f[j] = pack_f16x2(__uint_as_float(w[j] << 16) * f1 * f2,
                                              __uint_as_float(w[j] & 0xffff0000u) * f1 * f2);
                        *at = make_uint4(f[0], f[1], f[2], f[3]);
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(q_ready);
            }
            const int k1 = v.k1[h];
            for (int kt = v.k0[h]; kt < k1; ++kt, ++n) {
                const int key0 = kt * kKeyTile;
                float scale = row_scale;
                uint32_t refs = 0;
                if (kFp8) {  // what is known of this tile once its V has come, after its K
                    const uint32_t t = tiles + (uint32_t)(kt - it.k0);
                    wait(&ref_full[t % kRefs], t / kRefs & 1);
                    refs = tile_refs[t % kRefs];
                    // a row whose scores are all but 0 must not make -inf * 0 of the mask
                    scale = fmaxf(row_scale * pow2((int)(refs & 255) - 127), 0x1p-120f);
                }
                wait(&s_full[h], n & 1);
                tc::tc_fence_after();
                // The scores are read twice, for the maximum and for the probabilities, 32 columns at a time
                // in loops that stay rolled: tensor memory gives 128 columns in about 50 cycles, while code
                // for all of them is fetched slower than it runs once other warps' code lies between
                // (e4m3, unrolled: 2470 us, rolled 1790; bf16 the same; 8192 rows over 16384 tokens).
                const bool edge = key0 < lo_all || key0 + kKeyTile > hi_all;
                uint32_t s[32];
                auto load = [&](int i) {
                    tc::tmem_ld32(ts + i * 32, s);
                    tc::tmem_wait_ld();
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int key = key0 + i * 32 + j;
                            if (key < lo || key >= hi) s[j] = 0xff800000u;
                        }
                    }
                };
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    load(i);
#pragma unroll
                    for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[j]));
                }
                const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale);
                const bool move = mn - m > kLoose;  // also from -inf
                const int v_ref = refs >> 8;  // 256 and more: far
                if (kt == v.k0[h] && (!kFp8 || v_ref < 256)) {
                    m = mn;
                    o_ref = v_ref;
                } else if (__any_sync(0xffffffffu, move || (kFp8 && v_ref != o_ref))) {
                    if (kFp8 && v_ref >= 256) {
                        // Scales far from each other: each thread does its row alone, in fp32, every key with its own
                        // scale.  Here, where few tiles come, and in little code: the loops around it lose by
                        // every instruction between them (a form on the MMAs, with bf16 values, from a branch of
                        // its own: 166 us for ragged chunks whose scales are near, 162 with this).
                        const uint32_t t = tiles + (uint32_t)(kt - it.k0), entry = 2 * t + 1;
                        const uint8_t* sc = tile_scales + t % kRefs * (2 * kKeyTile);
                        const uint8_t* values = ring + entry % C::kEntries * C::kEntryBytes;
                        auto score = [&](uint32_t x, int j) {
                            const int key = key0 + j;
                            return key < lo || key >= hi ? -CUDART_INF_F : __uint_as_float(x) * row_scale * scale_of(sc[j]);
                        };
                        uint32_t x[8];
                        float top = m;
#pragma unroll 1
                        for (int i = 0; i < 16; ++i) {
                            tmem_ld8(ts + i * 8, x);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j) top = fmaxf(top, score(x[j], i * 8 + j));
                        }
                        const bool first = kt == v.k0[h];
                        float f = m == -CUDART_INF_F ? 1.0f : exp2_fast(m - top);
                        m = top;
                        l *= f;
                        if (!first) f *= pow2(o_ref - (v_ref & 255));
                        o_ref = v_ref & 255;
                        // the weights, in the place of the scores
                        const float from = m == -CUDART_INF_F ? 0.0f : m;
#pragma unroll 1
                        for (int i = 0; i < 16; ++i) {
                            tmem_ld8(ts + i * 8, x);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float w = exp2_fast(score(x[j], i * 8 + j) - from);
                                l += w;
                                x[j] = __float_as_uint(w * pow2((int)sc[kKeyTile + i * 8 + j] - o_ref + kPBits));
                            }
                            tmem_st8(ts + i * 8, x);
                        }
                        tmem_wait_st();
                        wait(&full[entry % C::kEntries], entry / C::kEntries & 1);
                        float add[kD];  // not in registers: indexed in a loop
#pragma unroll 1
                        for (int c = 0; c < kD / 8; ++c) {
                            float2 sum[4] = {};
#pragma unroll 1
                            for (int i = 0; i < 16; ++i) {
                                tmem_ld8(ts + i * 8, x);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const uint4 q = *reinterpret_cast<const uint4*>(
                                        values + (c >> 3) * C::kBlockBytes + (i * 8 + j) * 128 + (((c & 7) ^ j) << 4));
                                    const uint32_t codes[4] = {q.x, q.y, q.z, q.w};
                                    const float2 w = make_float2(__uint_as_float(x[j]), __uint_as_float(x[j]));
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        sum[y] = fma2(w, __half22float2(*reinterpret_cast<const __half2*>(&codes[y])), sum[y]);
                                }
                            }
#pragma unroll
                            for (int y = 0; y < 4; ++y) add[c * 8 + 2 * y] = sum[y].x, add[c * 8 + 2 * y + 1] = sum[y].y;
                        }
                        // the MMA adds nothing (or makes o zeros, if this tile is the first)
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = 0;
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) tmem_st8(ts + i * 8, x);
                        tmem_wait_st();
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&p_full[h]);
                        wait(&pv_done[h], n & 1);
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < kD / 8; ++i) {
                            tmem_ld8(to + i * 8, x);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                x[j] = __float_as_uint(fmaf(__uint_as_float(x[j]), f, add[i * 8 + j]));
                            tmem_st8(to + i * 8, x);
                        }
                        tmem_wait_st();
                        continue;
                    }
                    float f = move ? exp2_fast(m - mn) : 1.0f;
                    if (move) m = mn;
                    l *= f;
                    if (kFp8) {
                        f *= pow2(o_ref - v_ref);
                        o_ref = v_ref;
                    }
                    wait(&pv_done[h], (n - 1) & 1);
                    tc::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < kD / 16; ++i) {
                        uint32_t o[16];
                        tmem_ld16(to + i * 16, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st16(to + i * 16, o);
                    }
                }
                // e4m3: probabilities come out times 2^kPBits; the sum takes that back
                const float base = (m == -CUDART_INF_F ? 0.0f : m) - (kFp8 ? (float)kPBits : 0.0f);
                const float2 sc2 = make_float2(scale, scale), nb2 = make_float2(-base, -base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    load(i);
                    uint32_t out[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float2 x = make_float2(__uint_as_float(s[2*j]), __uint_as_float(s[2*j + 1]));
                        x = fma2(x, sc2, nb2);
                        x.x = exp2_fast(x.x);
                        x.y = exp2_fast(x.y);
                        sum[j & 1] = add2(sum[j & 1], x);
                        out[j] = kFp8 ? pack_f16x2(x.x, x.y) : cvt_bf16x2(x.x, x.y);
                    }
                    tmem_st16(ts + i * 16, out);
                }
                tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&p_full[h]);
                sum[0] = add2(sum[0], sum[1]);
                l += (sum[0].x + sum[0].y) * (kFp8 ? 1.0f / (1 << kPBits) : 1.0f);
            }
            // the item again, from the cursor: its fields would cost registers throughout the loop above
            __syncwarp();
            asm volatile("" ::: "memory");
            c = cursors[h];
            it = take(p, c);
            v = halves(p, it);
            const bool any = v.k0[h] < v.k1[h];
            if (any) {
                wait(&pv_done[h], (n - 1) & 1);
                tc::tc_fence_after();
            }
            tiles += it.n;
            const float o_unit = kFp8 ? pow2(o_ref - 127 - kPBits) : 1.0f;
            if (it.whole) {
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                uint16_t* out = p.o + at.token * p.o_ld + at.head * p.o_head;
#pragma unroll
                for (int i = 0; i < kD / 32; ++i) {
                    uint32_t o[32];
                    if (any) {
                        tc::tmem_ld32(to + i * 32, o);
                        tc::tmem_wait_ld();
                    }
                    if (valid) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                w[x] = l == 0.0f ? 0u  // in two steps: the product of the factors may be subnormal
                                                 : cvt_bf16x2(__uint_as_float(o[8 * j + 2 * x]) * inv * o_unit,
                                                              __uint_as_float(o[8 * j + 2 * x + 1]) * inv * o_unit);
                            *reinterpret_cast<uint4*>(out + i * 32 + j * 8) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (valid && p.lse)
                    p.lse[(int64_t)at.token * p.heads * p.group + at.head] =
                        l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
            } else {
                float down = 1.0f;
                if (kFp8) {
                    const int up = sum_exp(l);
                    down = pow2(-up);
                    m += (float)up;
                    l *= down;
                }
                // parts: [four columns][row], so that a warp's rows lie side by side
                const int slot = it.first ? 0 : 1, r = h * kHalfRows + row;
                float4* out = reinterpret_cast<float4*>(part_o(p, blockIdx.x, slot)) + r;
#pragma unroll
                for (int i = 0; i < kD / 32; ++i) {
                    uint32_t o[32];
                    if (any) {
                        tc::tmem_ld32(to + i * 32, o);
                        tc::tmem_wait_ld();
                    }
                    auto of = [&](int j) { return __uint_as_float(o[j]) * down * o_unit; };
                    if (valid) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            out[(i * 8 + j) * kMaxRows] = any ? make_float4(of(4 * j), of(4 * j + 1), of(4 * j + 2), of(4 * j + 3))
                                                              : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
                if (valid) part_ml(p, blockIdx.x, slot)[r] = make_float2(m, l);
                join<kD>(p, it, start, at, r, valid, &last_s, sync);
                sync();  // the flag may be written again
            }
            tc::tc_fence_before();  // o has been read: the next item's first arrival on p_full says so
            asm volatile("bar.sync %0, 128;" ::"r"(2 + h) : "memory");
            if ((threadIdx.x & 127) == 0) cursors[h] = c;
            asm volatile("bar.sync %0, 128;" ::"r"(2 + h) : "memory");
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) tc::tmem_dealloc(tmem, 512);
}

// q as (d, head, token): a box holds the rows of half a query tile in (token, group) order.
bool make_q_map(CUtensorMap* m, const Params& p, int head_dim, int half_tokens) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    const cuuint64_t heads = (cuuint64_t)p.heads * p.group;
    cuuint64_t dims[3] = {(cuuint64_t)head_dim, heads, (cuuint64_t)p.T};
    cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? p.q_head * 2 : head_dim * 2),
                             (cuuint64_t)(p.T > 1 ? p.q_ld * 2 : head_dim * 2)};
    cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)half_tokens};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kD, bool kFp8>
cudaError_t launch_as(const moe_kv_cache& c, const Params& p, int grid, cudaStream_t st) {
    CUtensorMap qm, km, vm;
    if (!make_q_map(&qm, p, kD, p.tokens_per_tile / 2) || !make_pool_map(&km, c, c.k) || !make_pool_map(&vm, c, c.v))
        return cudaErrorInvalidValue;
    auto kern = attn_tile_kernel<kD, kFp8>;
    constexpr int smem = Cfg<kD, kFp8>::kSmem;
    cudaError_t e = ensure_max_dynamic_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, Cfg<kD, kFp8>::kThreads, smem, st, p, qm, km, vm, c.k_scale, c.v_scale);
}

}  // namespace

cudaError_t launch_tiles(const moe_kv_cache& c, Params& p, int grid_cap, cudaStream_t st) {
    p.tokens_per_tile = 2 * (kHalfRows / p.group);
    // what a query tile costs beside its key tiles (1.7 us each) is about 7 us
    p.item_cost = 4;
    p.item_slack = 1;
    // a part costs its CTA and the joining one 2 us each and a join 2 more: with runs of at least 4 units
    // 128 rows over 500 tokens take 18 us, 24 with runs of 1, 22 of 6 (for the larger calls the same)
    p.cta_units = 4;
    const int grid = grid_for(p, grid_cap);
    const bool fp8 = c.dtype == MOE_FP8_E4M3;
    if (c.head_dim == 128)
        return fp8 ? launch_as<128, true>(c, p, grid, st) : launch_as<128, false>(c, p, grid, st);
    return fp8 ? launch_as<64, true>(c, p, grid, st) : launch_as<64, false>(c, p, grid, st);
}

}  // namespace attn
}  // namespace moe
