// Latent attention, expanded form, for prompts: every head has its own keys (128 numbers, and 64 that all heads
// share) and values (128).  Bound by the tensor cores; the pipeline is attn_tile.cuh's: a query tile is two
// halves of 128 rows (here tokens of one head) over the same key tiles, and while the softmax of one half
// runs, the tensor cores work on the other.  A prompt of 8192 tokens with 128 heads takes 1.87-2.11 ms from box to box,
// 1300-1470 TFLOP/s, and 2.20 once a busy GPU is at its power cap; ragged prompts of up to 1100 new tokens with 16 heads
// 85 us.
//   S = Q K^T    k = 192: 12 instructions of 128 rows x 128 keys      O += P V    8 of 128 rows x 128 columns
// Scores, probabilities and output fill tensor memory as there (S0 | S1 | O0 | O1, P over S).
//
// Q takes 96 KB, so the ring holds 128 KB, less than two key tiles (80 KB).  Its entries are 16 KB pieces, each
// given back by itself: a key tile's three blocks of 64 columns, and the halves of 64 keys of its values.  They
// arrive on one barrier for a tile's keys and one for its values: the issuing warp's waits, even those for what
// is there already, stand between the MMAs (a barrier for each piece: 2161 us where this took 2003).
//
// A pair of key tiles (both halves) takes 3800 cycles of the 2590 that its 40 MMAs last by themselves: shared memory
// is busy for 3200 (the MMAs' operands, the transposed ones at half rate, and the copies), and a half's chain of
// scores, softmax (2200 cycles, beside the other half's on the same schedulers) and product is 3700.
//
//   warps 0-3, 4-7   softmax and epilogue of half 0, 1 (a thread owns a row)
//   warp 8           issues the MMAs
//   warps 9-11       copies: keys, values, shared keys and Q (one warp took 800 cycles a piece, 4000 a key tile)
#include "attn_tile.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kKeyCols = 192, kValueCols = 128;
constexpr int kXThreads = 384;
constexpr int kPieceBytes = 16384;
constexpr int kHalfBytes = 3 * kHalfRows * 128;  // of Q
constexpr int kRingPieces = 8;
constexpr int kXBars = kRingPieces + 4 + 2 + 6 + 2;
constexpr int kXSmem = 1024 + 2 * kHalfBytes + kRingPieces * kPieceBytes + 8 * kXBars + 8;
static_assert(kXSmem <= 232448 - 512, "");

__global__ void __launch_bounds__(kXThreads, 1)
    attn_expanded_kernel(const __grid_constant__ DenseParams p, const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap rmap,
                         const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* qs = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);  // by an offset: accesses keep 32-bit addresses
    uint8_t* ring = qs + 2 * kHalfBytes;
    uint64_t* empty = reinterpret_cast<uint64_t*>(ring + kRingPieces * kPieceBytes);  // of each piece
    uint64_t* k_full = empty + kRingPieces;  // [2] of a tile's keys, by the tile's parity
    uint64_t* v_full = k_full + 2;           // [2] of its values
    uint64_t* q_full = v_full + 2;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;  // [2] scores of a half are in tensor memory
    uint64_t* p_full = s_full + 2;   // [2] its probabilities are
    uint64_t* pv_done = p_full + 2;  // [2] they have been multiplied into o
    uint64_t* done = pv_done + 2;
    uint64_t* never = done + 1;
    uint32_t* cmds = reinterpret_cast<uint32_t*>(never + 1);  // [2] of a key tile
    __shared__ Start start;
    __shared__ Cursor cursors[2];  // where the two softmax groups stand: not held in registers
    __shared__ int abort_s, last_s;
    __shared__ uint32_t tmem_s;
    volatile int* abort = &abort_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMmaWarp = 8, kCopyWarp = 9;
    if (threadIdx.x == 0) {
        abort_s = 0;
        for (int i = 0; i < kRingPieces; ++i) tc::mbar_init(&empty[i], 1);
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_empty, 1);
        for (int h = 0; h < 2; ++h) {
            tc::mbar_init(&k_full[h], 2);
            tc::mbar_init(&v_full[h], 1);
            tc::mbar_init(&s_full[h], 1);
            tc::mbar_init(&p_full[h], 4);
            tc::mbar_init(&pv_done[h], 1);
        }
        tc::mbar_init(done, 1);
        tc::mbar_init(never, 1);
        tc::fence_barrier_init();
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&rmap);
        tc::prefetch_tmap(&vmap);
    }
    __syncthreads();
    pdl_begin();
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&tmem_s, 512);
        tc::tmem_relinquish();
        tc::tc_fence_before();
    }
    locate<kXThreads>(p, reinterpret_cast<uint32_t*>(ring), &start);
    tc::tc_fence_after();
    const uint32_t tmem = tmem_s;
    if (p.inject_ns > 0 && blockIdx.x == 0) {  // test hook: the failure path of a bounded wait
        if (threadIdx.x == 0) {
            tc::wait_on_nothing(never, (uint64_t)p.inject_ns);
            set_err(p.err, MOE_ERR_TIMEOUT);
            let_go<kValueCols>(p, start, &last_s);
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
        regs_dec<120>();
        if (warp >= kCopyWarp) {
            // -------------------------------------------------------- copies
            // of a key tile's five pieces: 0 and 1 (keys), 3 and 4 (values), 2 (shared keys) and Q
            const int role = warp - kCopyWarp, b0 = role == 0 ? 0 : role == 1 ? 3 : 2, b1 = role == 2 ? 3 : b0 + 2;
            uint32_t tiles = 0, sent = 0, items = 0, q_sent = 0;
            while (more(cur)) {
                const Item it = take(p, cur);
                if (it.n == 0) continue;
                const Halves v = halves(p, it);
                const int row0 = it.r.row0 + it.tile * p.tokens_per_tile, key_row0 = p.cu_kv[it.b];
                if (role == 2) {
                    if (items > 0) wait(q_empty, (items - 1) & 1);
                    ++items;
                    if (!*abort) {
                        ++q_sent;
                        if (lane == 0) {
                            tc::mbar_arrive_expect_tx(q_full, v.count * kHalfBytes);
                            for (int h = 0; h < v.count; ++h)
                                for (int b = 0; b < 3; ++b)
                                    tc::tma_load_3d(qs + (h * 3 + b) * kHalfRows * 128, &qmap, q_full, b * 64, it.head,
                                                    row0 + h * kHalfRows);
                        }
                        __syncwarp();
                    }
                }
                for (int k = 0; k < it.n; ++k, ++tiles) {
                    const int kt = it.k0 + k, key0 = kt * kKeyTile, row = key_row0 + key0;
                    // (rows past the last key's are the next request's, or past the tensor: zeros)
#pragma unroll 1
                    for (int b = b0; b < b1; ++b) {
                        const uint32_t at = tiles * 5 + b, e = at % kRingPieces;
                        if (at >= kRingPieces) wait(&empty[e], (at / kRingPieces - 1) & 1);
                        if (b == 0) {
                            uint32_t cmd = (uint32_t)min(it.s.hi - key0, kKeyTile) << kSeenHi;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (active(v, h, kt)) cmd |= kAct0 << h | (kt == v.k0[h] ? kFirst0 << h : 0);
                            if (k == 0) cmd |= kNewQ;
                            if (k == it.n - 1) cmd |= kLastK;
                            if (lane == 0) cmds[tiles & 1] = cmd;
                        }
                        if (*abort) continue;
                        sent = tiles + 1;
                        if (lane == 0) {
                            uint8_t* dst = ring + e * kPieceBytes;
                            uint64_t* bar = role == 1 ? &v_full[tiles & 1] : &k_full[tiles & 1];
                            if (b == b0) tc::mbar_arrive_expect_tx(bar, (b1 - b0) * kPieceBytes);
                            if (b < 2) {
                                tc::tma_load_3d(dst, &kmap, bar, b * 64, it.head, row);
                            } else if (b == 2) {
                                tc::tma_load_2d(dst, &rmap, bar, 0, row);
                            } else {
                                tc::tma_load_3d(dst, &vmap, bar, 0, it.head, row + (b - 3) * 64);
                                tc::tma_load_3d(dst + kPieceBytes / 2, &vmap, bar, 64, it.head, row + (b - 3) * 64);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (*abort) {  // copies still in flight land (or a bounded wait gives up) before the CTA ends
                for (uint32_t t = sent, i = 0; t-- > 0 && i < 2; ++i)
                    tc::mbar_wait_bounded(role == 1 ? &v_full[t & 1] : &k_full[t & 1], t >> 1 & 1);
                if (q_sent > 0) tc::mbar_wait_bounded(q_full, (q_sent - 1) & 1);
            }
            if (role != 1) {
                const uint32_t at = tiles * 5;
                if (at >= kRingPieces) wait(&empty[at % kRingPieces], (at / kRingPieces - 1) & 1);
                if (lane == 0) {
                    if (role == 0) cmds[tiles & 1] = kStop;
                    tc::mbar_arrive(&k_full[tiles & 1]);
                }
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------- MMAs
            constexpr uint32_t kIdescS = tc::idesc_bf16_f32(128, kKeyTile);
            constexpr uint32_t kIdescO = tc::idesc_bf16_f32(128, kValueCols) | kIdescBMn;
            uint32_t at = 0;  // the next piece
            uint32_t tiles = 0, queries = 0, np0 = 0, np1 = 0;  // tiles: key tiles begun
            const uint64_t q_desc = tc::desc_sw128_kmajor(tc::smem_u32(qs));
            const uint64_t k_desc = tc::desc_sw128_kmajor(tc::smem_u32(ring));
            const uint64_t v_desc = desc_sw128_mnmajor(tc::smem_u32(ring), kPieceBytes / 2);
            auto commit = [&](uint64_t* bar) {
                if (tc::elect_one()) tc::mma_commit(bar);
                __syncwarp();
            };
            // S_h = Q_h K^T from the pieces at `first`; the last half to use them gives each back as it goes
            auto scores = [&](int h, uint32_t first, bool release) {
                if (tc::elect_one()) {
                    const uint64_t a = q_desc + (uint32_t)(h * (kHalfBytes >> 4));
#pragma unroll
                    for (int b = 0; b < 3; ++b) {
                        const uint64_t k = k_desc + (first + b) % kRingPieces * (kPieceBytes >> 4);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            tc::mma_bf16(tmem + h * 128, a + b * (kHalfRows * 128 >> 4) + s * 2, k + s * 2, kIdescS,
                                         b + s > 0);
                        if (release) tc::mma_commit(&empty[(first + b) % kRingPieces]);
                    }
                    tc::mma_commit(&s_full[h]);
                }
                __syncwarp();
            };
            auto values = [&](int h, uint32_t first, uint32_t accumulate, bool release) {  // O_h (+)= P_h V
                if (tc::elect_one()) {
#pragma unroll
                    for (int s = 0; s < kKeyTile / 16; ++s) {
                        mma_bf16_ta(tmem + 256 + h * 128, tmem + h * 128 + s * 8,
                                    v_desc + (first + s / 4) % kRingPieces * (kPieceBytes >> 4) + s % 4 * (2048 >> 4),
                                    kIdescO, s > 0 ? 1u : accumulate);
                        if (release && s % 4 == 3) tc::mma_commit(&empty[(first + s / 4) % kRingPieces]);
                    }
                    tc::mma_commit(&pv_done[h]);
                }
                __syncwarp();
            };
            // the key tile at `at` is there: its command, with Q there too
            auto keys = [&]() -> uint32_t {
                wait(&k_full[tiles & 1], tiles >> 1 & 1);
                const uint32_t cmd = cmds[tiles & 1];
                if (cmd & kStop) return cmd;
                if (cmd & kNewQ) wait(q_full, queries++ & 1);
                tc::tc_fence_after();
                return cmd;
            };
            auto keys_done = [&](uint32_t cmd) {
                if (cmd & kLastK) commit(q_empty);
                ++tiles;
                at += 3;
            };
            uint32_t cmd = keys();
            if (!(cmd & kStop)) {
                if (cmd & kAct0) scores(0, at, !(cmd & (kAct0 << 1)));
                if (cmd & (kAct0 << 1)) scores(1, at, true);
                keys_done(cmd);
            }
            while (!(cmd & kStop)) {
                const uint32_t va = at;
                at += 2;
                wait(&v_full[(tiles - 1) & 1], (tiles - 1) >> 1 & 1);
                const int z1 = cmd >> kSeenHi & 255;
                if (z1 < kKeyTile) {
                    // what lies behind the request's keys may be anything, NaN among it: 0 * NaN would reach o
                    for (int i = lane + z1 * 16; i < kKeyTile * 16; i += 32) {
                        const int key = i >> 4;
                        reinterpret_cast<uint4*>(ring + (va + (key >> 6)) % kRingPieces * kPieceBytes +
                                                 (i >> 3 & 1) * (kPieceBytes / 2))[(key & 63) * 8 + (i & 7)] =
                            make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                // within a query tile the next scores of a half follow its product at once; those of
                // another query tile wait for its rows, and both halves' products come first
                const bool last = cmd & kLastK;
                uint32_t then = 0;
                if (cmd & kAct0) {
                    wait(&p_full[0], np0++ & 1);
                    tc::tc_fence_after();
                    values(0, va, cmd & kFirst0 ? 0 : 1, !(cmd & (kAct0 << 1)));
                }
                if (!last) {
                    then = keys();
                    if (then & kAct0) scores(0, at, !(then & (kAct0 << 1)));
                }
                if (cmd & (kAct0 << 1)) {
                    wait(&p_full[1], np1++ & 1);
                    tc::tc_fence_after();
                    values(1, va, cmd & (kFirst0 << 1) ? 0 : 1, true);
                }
                if (last) {
                    then = keys();
                    if (then & kAct0) scores(0, at, !(then & (kAct0 << 1)));
                }
                if (then & (kAct0 << 1)) scores(1, at, true);
                if (!(then & kStop)) keys_done(then);
                cmd = then;
            }
            commit(done);
            tc::mbar_wait_bounded(done, 0);
        }
    } else {
        // ------------------------------------------------------------ softmax and epilogue
        regs_inc<192>();
        const int h = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter of the lanes
        const uint32_t ts = tmem + h * 128 + lanes, to = tmem + 256 + h * 128 + lanes;
        auto sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        uint32_t n = 0;  // key tiles of this half so far
        for (;;) {
            Cursor c = cursors[h];
            if (!more(c)) break;
            Item it = take(p, c);
            Halves v = halves(p, it);
            const int q = h * kHalfRows + row;  // row of the query tile
            const bool valid = q < it.tokens;
            const int pos0 = it.r.kv - it.r.n + it.tile * p.tokens_per_tile + h * kHalfRows;
            const int hi = !valid ? 0 : p.causal ? min(pos0 + row + 1, it.r.kv) : it.r.kv;
            const int hi_all = p.causal ? min(it.r.kv, pos0 + 1) : it.r.kv;  // every row of the half sees keys below
            float m = -CUDART_INF_F, l = 0.0f;                              // m in powers of two
            const int k1 = v.k1[h];
            for (int kt = v.k0[h]; kt < k1; ++kt, ++n) {
                const int key0 = kt * kKeyTile;
                wait(&s_full[h], n & 1);
                tc::tc_fence_after();
                // read twice, in rolled loops, as in attn_tile.cuh
                const bool edge = key0 + kKeyTile > hi_all;
                uint32_t s[32];
                auto load = [&](int i) {
                    tc::tmem_ld32(ts + i * 32, s);
                    tc::tmem_wait_ld();
                    if (edge) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (key0 + i * 32 + j >= hi) s[j] = 0xff800000u;
                    }
                };
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    load(i);
#pragma unroll
                    for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[j]));
                }
                const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2);
                const bool move = valid && mn - m > kLoose;  // also from -inf
                if (kt == v.k0[h]) {
                    m = mn;
                } else if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? exp2_fast(m - mn) : 1.0f;
                    if (move) m = mn;
                    l *= f;
                    wait(&pv_done[h], (n - 1) & 1);
                    tc::tc_fence_after();
#pragma unroll
                    for (int i = 0; i < kValueCols / 16; ++i) {
                        uint32_t o[16];
                        tmem_ld16(to + i * 16, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st16(to + i * 16, o);
                    }
                }
                const float base = m == -CUDART_INF_F ? 0.0f : m;
                const float2 nb2 = make_float2(-base, -base);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    load(i);
                    uint32_t out[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float2 x = make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
                        x = fma2(x, sc2, nb2);
                        x.x = exp2_fast(x.x);
                        x.y = exp2_fast(x.y);
                        sum[j & 1] = add2(sum[j & 1], x);
                        out[j] = cvt_bf16x2(x.x, x.y);
                    }
                    tmem_st16(ts + i * 16, out);
                }
                tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&p_full[h]);
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
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
            const RowAt at = {it.r.row0 + it.tile * p.tokens_per_tile + q, it.head};
            if (it.whole) {
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                uint16_t* out = p.o + at.token * p.o_ld + at.head * p.o_head;
#pragma unroll
                for (int i = 0; i < kValueCols / 32; ++i) {
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
                                w[x] = l == 0.0f ? 0u
                                                 : cvt_bf16x2(__uint_as_float(o[8 * j + 2 * x]) * inv,
                                                              __uint_as_float(o[8 * j + 2 * x + 1]) * inv);
                            *reinterpret_cast<uint4*>(out + i * 32 + j * 8) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (valid && p.lse)
                    p.lse[(int64_t)at.token * p.heads + at.head] =
                        l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
            } else {
                // parts: [four columns][row], so that a warp's rows lie side by side
                const int slot = it.first ? 0 : 1;
                float4* out = reinterpret_cast<float4*>(part_o(p, blockIdx.x, slot)) + q;
#pragma unroll
                for (int i = 0; i < kValueCols / 32; ++i) {
                    uint32_t o[32];
                    if (any) {
                        tc::tmem_ld32(to + i * 32, o);
                        tc::tmem_wait_ld();
                    }
                    if (valid) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            out[(i * 8 + j) * kMaxRows] =
                                any ? make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                  __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
                if (valid) part_ml(p, blockIdx.x, slot)[q] = make_float2(m, l);
                join<kValueCols>(p, it, start, at, q, valid, &last_s, sync);
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

// Rows of `cols` numbers as (d, head, row), boxes of 64 columns of `rows` rows of one head.  The stride of an
// index with one value is not used, and may be any number.
bool make_rows_map(CUtensorMap* m, const void* base, int cols, int heads, int rows_all, int64_t head_stride, int64_t ld,
                   int rows) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows_all};
    cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? head_stride * 2 : cols * 2),
                             (cuuint64_t)(rows_all > 1 ? ld * 2 : cols * 2)};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool make_rope_map(CUtensorMap* m, const moe_attn_expanded_args& a) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tma_encode_fn());
    if (!enc) return false;
    cuuint64_t dims[2] = {64, (cuuint64_t)a.S};
    cuuint64_t strides[1] = {(cuuint64_t)(a.S > 1 ? a.rope_ld * 2 : 128)};
    cuuint32_t box[2] = {64, kKeyTile};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.k_rope), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_expanded(const moe_attn_expanded_args& a, int grid_cap, cudaStream_t st) {
    using namespace attn;
    DenseParams p = {};
    p.q = static_cast<const uint16_t*>(a.q);
    p.o = static_cast<uint16_t*>(a.o);
    p.lse = a.lse;
    p.o_ld = a.o_ld;
    p.o_head = a.o_head_stride;
    p.cu_q = a.cu_q;
    p.cu_kv = a.cu_kv;
    p.T = a.T;
    p.S = a.S;
    p.B = a.B;
    p.max_q = a.max_q;
    p.max_kv = a.max_kv;
    p.heads = a.num_heads;
    p.group = 1;
    p.tokens_per_tile = 2 * kHalfRows;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.causal = a.causal;
    p.err = a.err_flag;
    p.counters = static_cast<uint32_t*>(a.workspace);
    p.parts = static_cast<uint8_t*>(a.workspace) + kMaxCtas * sizeof(uint32_t);
    p.inject_ns = wait_injection_ns();
    // a query tile costs about two key tiles (2 us each) beside its own; runs of at least 4 units as in attn_tile.cuh
    p.item_cost = 2;
    p.item_slack = 1;
    p.cta_units = 4;
    CUtensorMap qm, km, rm, vm;
    if (!make_rows_map(&qm, a.q, kKeyCols, a.num_heads, a.T, a.q_head_stride, a.q_ld, kHalfRows))
        return cudaErrorInvalidValue;
    km = rm = vm = qm;  // no keys at all: no copies from them
    if (a.S > 0 && (!make_rows_map(&km, a.k, 128, a.num_heads, a.S, a.k_head_stride, a.k_ld, kKeyTile) ||
                    !make_rows_map(&vm, a.v, 128, a.num_heads, a.S, a.v_head_stride, a.v_ld, kKeyTile / 2) ||
                    !make_rope_map(&rm, a)))
        return cudaErrorInvalidValue;
    auto kern = attn_expanded_kernel;
    cudaError_t e = ensure_max_dynamic_smem(kern, kXSmem);
    if (e != cudaSuccess) return e;
    if (grid_cap > kMaxCtas) grid_cap = kMaxCtas;
    return launch_pdl(kern, grid_for(p, grid_cap), kXThreads, kXSmem, st, p, qm, km, rm, vm);
}

}  // namespace moe
