// What the paged attention's kernels share: how the work is cut and handed out, and how a
// query tile whose keys were shared out over several CTAs is put together.
//
// Rows.  For one key/value head, a request's queries are (token, group) rows, group fastest:
// the query heads that read the same keys sit in one tile, so the keys are read once for
// all of them.  A query tile holds tokens_per_tile tokens of one request.
//
// Units.  A unit is one query tile against one tile of kKeyTile keys; masked-out key tiles
// (after the causal diagonal, before the window) are no units, and a query tile that sees
// no key at all counts as one.  What a query tile takes beside its key tiles (its rows, its
// output, the pipeline's turn) stands in front of them as item_cost units more.  Units are
// numbered request by request, head by head, query tile by query tile, key tile by key tile,
// and each of N CTAs, the grid or U / cta_units if that is less, takes a run of U/N of them, rounded
// up for the first U mod N: ragged lengths cost no balance, and few rows over a long context are split over
// the whole GPU by the same rule that gives a CTA many short requests.  A boundary that falls
// into a tile's item_cost, or leaves fewer than item_slack of its units, moves to the tile's
// edge: no part of a tile is without keys, and none costs more than it spares.  Every CTA
// derives its two boundaries from the lengths on the device, so nothing is read back.
//
// Joining.  A query tile whose units span CTAs c0 < .. < c1 is finished by the last of them
// to arrive: each stores its part (unnormalised o, running maximum, sum) in its own slot of
// the workspace, then counts itself in one of the tile's counters; the last sums the parts in CTA
// order, so the result does not depend on who came last.  It also clears the counter for the
// next call.  (Large parts are summed a few at a time in the same way.)  A counter is that of a
// CTA that continues the tile; a CTA continues no other.
#pragma once

#include <math_constants.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace moe {
namespace tc {

// 4-D tiled load of the box at (c0 innermost, c1, c2, c3); completion is signalled on `bar` as
// transaction bytes.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, "
        "%6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// The same with a cache policy.  Of data that is read once, L2 gives the lines up before others.
__device__ __forceinline__ uint64_t policy_of(bool read_once) {
    uint64_t p;
    if (read_once)
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    else
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                                                 int c3, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, "
        "%4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}

// True in one lane of a converged warp: the form in which single-thread instructions
// (tcgen05.mma, its commit) are best issued, since the rest of the warp stays uniform.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

}  // namespace tc

namespace attn {

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
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

constexpr int kKeyTile = 128;
constexpr int kMaxCtas = 1024;     // counters at the front of the workspace
constexpr int kMaxRows = 256;      // rows of the largest query tile

// One part of a split tile: o (rows x head_dim, in the kernel's own order), then [rows] (max, sum).
constexpr size_t kPartBytes = (size_t)kMaxRows * 128 * 4 + (size_t)kMaxRows * 8;

struct Params {
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    int64_t q_ld, q_head, o_ld, o_head;
    const int32_t* cu_q;
    const int32_t* kv_len;
    const int32_t* table;
    int table_ld;
    int T, B, max_q, max_kv;
    int heads, group;         // key/value heads; query heads per key/value head
    int tokens_per_tile;
    int num_pages, page_shift, page_size;
    float scale_log2;         // scale * log2(e): scores in powers of two
    int causal, window;
    int item_cost, item_slack, cta_units;  // in units
    int32_t* err;
    uint32_t* counters;       // [kMaxCtas], all zero between calls
    uint8_t* parts;           // [grid][2] parts: slot 0 the tile begun last, slot 1 the tile continued
    int64_t inject_ns;
    const uint64_t* tree;     // of a tree of drafted tokens: a new token's branch, else null
};

// A request's lengths; n = 0 for one that is refused (its rows are not written).
struct Request {
    int row0, n, kv;
};

__device__ __forceinline__ Request request(const Params& p, int b, bool report) {
    Request r;
    r.row0 = p.cu_q[b];
    r.n = p.cu_q[b + 1] - r.row0;
    r.kv = p.kv_len[b];
    const int64_t room = (int64_t)p.table_ld << p.page_shift;
    if (r.row0 < 0 || r.n < 0 || r.n > p.max_q || r.row0 > p.T - r.n || r.kv < 0 || r.kv > p.max_kv || r.kv > room) {
        if (report) set_err(p.err, MOE_ERR_BAD_INDEX);
        r.n = 0;
    }
    return r;
}

// Keys in packed rows (moe_attn_expanded) instead of pages: request b's are cu_kv[b] .. cu_kv[b+1].  kv_len
// and the table are not used.
struct DenseParams : Params {
    const int32_t* cu_kv;
    int S;  // rows of keys
};
__device__ __forceinline__ Request request(const DenseParams& p, int b, bool report) {
    Request r;
    r.row0 = p.cu_q[b];
    r.n = p.cu_q[b + 1] - r.row0;
    const int first = p.cu_kv[b];
    r.kv = p.cu_kv[b + 1] - first;
    if (r.row0 < 0 || r.n < 0 || r.n > p.max_q || r.row0 > p.T - r.n || first < 0 || r.kv < 0 || r.kv > p.max_kv ||
        first > p.S - r.kv) {
        if (report) set_err(p.err, MOE_ERR_BAD_INDEX);
        r.n = 0;
    }
    return r;
}

// Key tiles [k0, k1) that query tile i of a request sees, and the keys [lo, hi) among them.
struct Span {
    int lo, hi, k0, units;
};
__device__ __forceinline__ Span span(const Params& p, const Request& r, int i) {
    Span s;
    const int t0 = i * p.tokens_per_tile, t1 = min(t0 + p.tokens_per_tile, r.n);
    s.hi = p.causal ? min(r.kv, max(r.kv - r.n + t1, 0)) : r.kv;
    s.lo = p.window > 0 ? max(0, r.kv - r.n + t0 - p.window + 1) : 0;
    s.k0 = s.lo / kKeyTile;
    s.units = s.hi > s.lo ? (s.hi + kKeyTile - 1) / kKeyTile - s.k0 : 0;
    return s;
}
__device__ __forceinline__ int tiles_of(const Params& p, const Request& r) {
    return (r.n + p.tokens_per_tile - 1) / p.tokens_per_tile;
}

// Where a CTA stands: a query tile and how many of its units lie before and inside the
// CTA's range.
struct Cursor {
    int b, head, tile;
    int unit;           // number of the tile's unit that comes first in this CTA's range
    int end;            // of the CTA's range
    int skip;           // units of the tile before `unit`, item_cost among them
    bool done;          // the tile has been taken: take() moves on first
    Request r;
};

// The tile that a CTA's boundary falls into.
struct Spot {
    int b, head, tile;
    int off, cost;  // units of the tile before the boundary, and all of them, item_cost among them
    Request r;
};
struct Start {  // in shared memory, filled by locate()
    Spot spot[2];    // of the CTA's first unit and of the one past its last
    int unit, end;   // its range, boundaries moved
    bool next;       // it begins at the tile after spot[0]'s
    int each, more;  // units of a CTA; the first `more` CTAs have one more
};

// The CTA whose unmoved range has unit u.
__device__ __forceinline__ int cta_of(const Start& st, int u) {
    const uint32_t first = (uint32_t)st.more * (st.each + 1), v = (uint32_t)u;
    return v < first ? v / (st.each + 1) : st.more + (v - first) / st.each;
}
__device__ __forceinline__ uint32_t cost_of(const Params& p, int units) {
    return (uint32_t)(max(1, units) + p.item_cost);
}

__device__ __forceinline__ uint32_t warp_incl(uint32_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// CTAs that get units, at least one each: no CTA has too few to be worth a part.
__device__ __forceinline__ uint32_t ctas_for(const Params& p, uint32_t total, uint32_t ctas) {
    return total == 0 ? 0 : min(ctas, max(total / (uint32_t)p.cta_units, 1u));
}

// Whole CTA (kThreads threads): the range of units of CTA `me` of `ctas` (here the CTA itself of the grid, or
// a team of CTAs that share a range) and the query tile it begins in.
// scratch: shared, p.B + 32 uint32, free again for copies after it.  Ends with a barrier;
// st->unit == st->end: nothing to do.
template <int kThreads, typename P>
__device__ void locate(const P& p, uint32_t* scratch, Start* st, uint32_t me = blockIdx.x,
                       uint32_t ctas = gridDim.x) {
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool single = p.max_q <= p.tokens_per_tile;  // one query tile a request
    if (single && p.B <= 32) {
        // a small batch, whose call is mostly this and other latencies: one warp, one barrier
        if (warp == 0) {
            Request r = {0, 0, 0};
            uint32_t one = 0;
            if (lane < p.B) {
                r = request(p, lane, me == 0);
                if (r.n > 0) one = cost_of(p, span(p, r, 0).units);
            }
            const uint32_t k = one * (uint32_t)p.heads, upto = warp_incl(k), at = upto - k;
            const uint32_t total = __shfl_sync(0xffffffffu, upto, 31);
            const uint32_t n = ctas_for(p, total, ctas);
            const uint32_t each = n ? total / n : 0, rest = n ? total - each * n : 0;
            int moved[2];
            bool next = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u = me + i < n ? (me + i) * each + min(me + i, rest) : total;
                moved[i] = (int)u;
                const uint32_t mine = __ballot_sync(0xffffffffu, u < total && u >= at && u < upto);
                if (mine == 0) continue;
                const int b = __ffs(mine) - 1;
                const uint32_t cost = __shfl_sync(0xffffffffu, one, b), in = u - __shfl_sync(0xffffffffu, at, b);
                int off = (int)(in % cost);
                if (off <= p.item_cost) {
                    moved[i] -= off;
                    off = 0;
                } else if (off >= (int)cost - p.item_slack) {
                    moved[i] += (int)cost - off;
                    if (i == 0) next = true;
                }
                if (i == 0) {
                    const int row0 = __shfl_sync(0xffffffffu, r.row0, b), rows = __shfl_sync(0xffffffffu, r.n, b);
                    const int kv = __shfl_sync(0xffffffffu, r.kv, b);
                    if (lane == 0) st->spot[0] = Spot{b, (int)(in / cost), 0, off, (int)cost, {row0, rows, kv}};
                }
            }
            if (lane == 0) {
                st->unit = moved[0];
                st->end = moved[1];
                st->next = next;
                st->each = (int)each;
                st->more = (int)rest;
            }
        }
        __syncthreads();
        return;
    }
    uint32_t* per = scratch + 32;  // units of one head of request b, unless a thread has one request
    const int run = (p.B + kThreads - 1) / kThreads;  // requests per thread, consecutive
    const int b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
    uint32_t mine = 0;
    Request r = {0, 0, 0};
    if (single) {
        for (int b = b0; b < b1; ++b) {
            r = request(p, b, me == 0);
            const uint32_t u = r.n > 0 ? cost_of(p, span(p, r, 0).units) : 0u;
            if (run > 1) per[b] = u;
            mine += u;
        }
    } else {
        for (int b = warp; b < p.B; b += kWarps) {
            const Request q = request(p, b, me == 0 && lane == 0);
            const int n = tiles_of(p, q);
            uint32_t s = 0;
            for (int i = lane; i < n; i += 32) s += cost_of(p, span(p, q, i).units);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) per[b] = s;
        }
        __syncthreads();
        for (int b = b0; b < b1; ++b) mine += per[b];
    }
    const uint32_t incl = warp_incl(mine);
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scratch[w];
        all += scratch[w];
    }
    const uint32_t total = all * (uint32_t)p.heads;  // host: below 2^31
    // no CTA's range is empty (before boundaries move) but those of surplus CTAs: the CTAs of a
    // split tile are consecutive
    const uint32_t n = ctas_for(p, total, ctas);
    const uint32_t each = n ? total / n : 0, rest = n ? total - each * n : 0;
    const uint32_t u[2] = {me < n ? me * each + min(me, rest) : total,
                           me + 1 < n ? (me + 1) * each + min(me + 1, rest) : total};
    const uint32_t at0 = (before + incl - mine) * (uint32_t)p.heads;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (u[i] >= total || u[i] < at0 || u[i] >= at0 + mine * (uint32_t)p.heads) continue;
        uint32_t at = at0;
        for (int b = b0; b < b1; ++b) {
            const uint32_t one = single && run == 1 ? mine : per[b], k = one * (uint32_t)p.heads;
            if (u[i] < at + k) {
                Spot& s = st->spot[i];
                s.b = b;
                s.head = (int)((u[i] - at) / one);
                s.tile = 0;
                s.off = (int)((u[i] - at) % one);  // units of this head's tiles before it
                s.cost = (int)one;
                s.r = single && run == 1 ? r : request(p, b, false);
                break;
            }
            at += k;
        }
    }
    __syncthreads();
    if (!single) {
        if (warp < 2 && u[warp & 1] < total) {
            Spot& s = st->spot[warp];
            const Request q = s.r;
            const int tiles = tiles_of(p, q);
            uint32_t left = (uint32_t)s.off;
            __syncwarp();
            for (int i0 = 0; i0 < tiles; i0 += 32) {
                const uint32_t c = i0 + lane < tiles ? cost_of(p, span(p, q, i0 + lane).units) : 0u;
                const uint32_t in = warp_incl(c);
                const uint32_t over = __ballot_sync(0xffffffffu, in > left);
                if (over) {
                    if (lane == __ffs(over) - 1) {
                        s.tile = i0 + lane;
                        s.off = (int)(left - (in - c));
                        s.cost = (int)c;
                    }
                    break;
                }
                left -= __shfl_sync(0xffffffffu, in, 31);
            }
        }
        __syncthreads();
    }
    if (tid == 0) {
        int moved[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            moved[i] = (int)u[i];
            if (i == 0) st->next = false;
            if (u[i] >= total) continue;
            const Spot& s = st->spot[i];
            if (s.off <= p.item_cost) {
                moved[i] -= s.off;
                if (i == 0) st->spot[0].off = 0;
            } else if (s.off >= s.cost - p.item_slack) {
                moved[i] += s.cost - s.off;
                if (i == 0) st->next = true;
            }
        }
        st->unit = moved[0];
        st->end = moved[1];
        st->each = (int)each;
        st->more = (int)rest;
    }
    tc::fence_proxy_async_smem();  // the scratch may become copies' destination
    __syncthreads();
}

__device__ __forceinline__ Cursor cursor(const Start& st) {
    Cursor c;
    c.b = st.spot[0].b;
    c.head = st.spot[0].head;
    c.tile = st.spot[0].tile;
    c.skip = st.spot[0].off;
    c.r = st.spot[0].r;
    c.unit = st.unit;
    c.end = st.end;
    c.done = st.next;
    return c;
}

// One stretch of work: a query tile and this CTA's units of it.
struct Item {
    int b, head, tile;
    Request r;
    Span s;
    int k0, n;          // first key tile and number of key tiles (0: the tile sees no key)
    int tokens;         // tokens of the query tile
    bool whole;         // no other CTA has units of this tile
    bool first;         // this CTA has the tile's first unit
    int tile_unit;      // number of the tile's first unit
    int cost;           // the tile's units, item_cost among them
};

__device__ __forceinline__ bool more(const Cursor& c) { return c.unit < c.end; }

// The next item.  The cursor moves to it only now: the lengths of a request are not waited
// for before its turn.
template <typename P>
__device__ __forceinline__ Item take(const P& p, Cursor& c) {
    if (c.done) {
        c.skip = 0;
        if (++c.tile >= tiles_of(p, c.r)) {
            c.tile = 0;
            if (++c.head >= p.heads) {
                c.head = 0;
                do {  // the range ends before the requests do
                    c.r = request(p, ++c.b, false);
                } while (c.r.n == 0);
            }
        }
    }
    Item it;
    it.b = c.b;
    it.head = c.head;
    it.tile = c.tile;
    it.r = c.r;
    it.s = span(p, c.r, c.tile);
    it.cost = (int)cost_of(p, it.s.units);
    it.tile_unit = c.unit - c.skip;
    const int n = min(it.cost - c.skip, c.end - c.unit);  // past item_cost: boundaries were moved
    it.first = c.skip == 0;
    it.whole = n == it.cost;
    it.k0 = it.s.k0 + (it.first ? 0 : c.skip - p.item_cost);
    it.n = it.s.units ? n - (it.first ? p.item_cost : 0) : 0;
    it.tokens = min(p.tokens_per_tile, c.r.n - c.tile * p.tokens_per_tile);
    c.unit += n;
    c.done = true;
    return it;
}

// The copying warp's view of an item's pages: lane i holds table entry first + i of 32, the
// next 32 are on their way, and so are the next item's first ones, so that no tile waits for
// its table entries (a load from the table takes longer than a tile's copies may).
struct Pages {
    int first, now, then;
};
__device__ __forceinline__ int page_entry(const Params& p, const Item& it, int i) {
    const bool in = it.n > 0 && i >= it.s.lo >> p.page_shift && ((int64_t)i << p.page_shift) < it.s.hi;
    return in ? __ldg(p.table + (int64_t)it.b * p.table_ld + i) : 0;
}
__device__ __forceinline__ Pages pages_of(const Params& p, const Item& it) {
    Pages g;
    const int lane = threadIdx.x & 31;
    g.first = (it.k0 * kKeyTile >> p.page_shift) & ~31;
    g.now = page_entry(p, it, g.first + lane);
    g.then = page_entry(p, it, g.first + 32 + lane);
    return g;
}
// The pages of a tile's boxes: lane i gets that of box row `pg` of the tile at key0 (the whole
// warp calls this; a tile's pages lie in one run of 32).
__device__ __forceinline__ int page_of(const Params& p, const Item& it, Pages& g, int key0, int pg) {
    const int i0 = key0 >> p.page_shift;
    if (i0 >= g.first + 32) {
        g.first += 32;
        g.now = g.then;
        g.then = page_entry(p, it, g.first + 32 + (threadIdx.x & 31));
    }
    return __shfl_sync(0xffffffffu, g.now, (i0 - g.first + pg) & 31);
}

// A tree of drafted tokens (moe_attn_tree): a row sees the tokens before its request's new ones and, of
// those, its branch: new token j stands at position first + j.  No bits past the request's tokens.
struct Branch {
    int first;
    uint64_t bits;
    __device__ __forceinline__ bool sees(int key) const { return key < first || (bits >> (key - first) & 1); }
    // bit j: whether it sees key + j.  A tile's mask from these costs a test a key; from sees(), 64-bit shifts in
    // both passes over the scores, trees of up to 64 nodes over 32 requests took 174 us instead of 106.
    __device__ __forceinline__ uint32_t word(int key) const {
        const int d = key - first;
        if (d >= 0) return d < 64 ? (uint32_t)(bits >> d) : 0u;
        return d > -32 ? (uint32_t)(bits << -d) | ((1u << -d) - 1) : 0xffffffffu;
    }
};
__device__ __forceinline__ Branch branch_of(const Params& p, const Request& r, int token) {
    const uint64_t bits = __ldg(p.tree + token) | 1ull << (token - r.row0);
    return {r.kv - r.n, r.n < 64 ? bits & ((1ull << r.n) - 1) : bits};
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e as a float, 0 below its normal range.
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.0f : __int_as_float((min(e, 127) + 127) << 23); }

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
// The power of two that brings a row whose largest magnitude has the bf16 bits mx into
// [2^14, 2^15), at most 2^100 (a row of zeros, or of numbers so small that its scores are 0).
__device__ __forceinline__ int f16_row_exp(uint32_t mx) { return min(14 - ((int)(mx >> 7) - 127), 100); }

// An e4m3 cache's value scales.  A weight is its probability times 2^(b - ref) and 2^kPBits, b the value's
// scale byte, ref a reference to which o refers as well.  In fp16 what a weight adds to o is off by 2^-11 of
// itself or by 2^-32 of a value at the reference, whichever is more; so fp16 takes the keys whose
// scales lie from the smallest one so far to 2^kNear above it, where the latter is 2^-20 of what any key
// may add.  Keys with larger values (and all of them, once values 2^60 larger have held the reference up) take
// a way whose weights keep their exponents: what a row gets from its keys does not depend on how
// large a value beside them is, one that the row hardly weighs or does not see.
constexpr int kPBits = 7;
constexpr uint32_t kNear = 12;
constexpr uint32_t kFarUp = 60;  // the most that a value's scale is above the reference: o stays in fp32's range
struct Scales {
    uint32_t lo, ref, top;  // smallest scale byte so far, reference, largest; top = 0: none yet
    uint32_t span;          // bytes from ref - span to ref change nothing here and are near the reference
};
// Whether scale bytes from lo to top are multiplied in fp16.
__device__ __forceinline__ bool near_ref(const Scales& w, uint32_t lo, uint32_t top) {
    return top <= w.ref && w.ref - lo <= kNear;
}
// Takes the scale bytes from lo to top in.
__device__ __forceinline__ void take_in(Scales& w, uint32_t lo, uint32_t top) {
    if (lo > top) return;  // none
    w.lo = w.top == 0 ? lo : min(w.lo, lo);
    w.top = max(w.top, top);
    w.ref = max(min(w.top, w.lo + kNear), w.top - min(w.top, kFarUp));
    w.span = min(w.ref - w.lo, kNear);
}
// Two e4m3 codes as fp16 -> as bf16 (exact).
__device__ __forceinline__ uint32_t f16x2_bf16x2(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16x2(f.x, f.y);
}
constexpr float kLoose = 8.0f;  // log2 of how far a row's maximum may run ahead of the one in use

// The exponent e by which a sum l of probabilities (relative to a maximum m that is followed loosely), o and m
// change to l 2^-e, o 2^-e and m + e before o, whose values may be near the end of fp32's range, is added up with
// others: l 2^-e is at most 2^-8, so 256 such o may be added.
__device__ __forceinline__ int sum_exp(float l) {
    const int e = (__float_as_int(l) >> 23) & 255;
    return e == 0 || e == 255 ? 0 : e - 127 + 9;
}

// The value of a UE8M0 scale byte (0: 2^-127, 255: NaN).
__device__ __forceinline__ float scale_of(uint8_t b) {
    return b == 255 ? CUDART_NAN_F : __uint_as_float(b == 0 ? 0x00400000u : (uint32_t)b << 23);
}

__device__ __forceinline__ float* part_o(const Params& p, int cta, int slot) {
    return reinterpret_cast<float*>(p.parts + ((size_t)cta * 2 + slot) * kPartBytes);
}
__device__ __forceinline__ float2* part_ml(const Params& p, int cta, int slot) {
    return reinterpret_cast<float2*>(p.parts + ((size_t)cta * 2 + slot) * kPartBytes + (size_t)kMaxRows * 128 * 4);
}

// Row r of a query tile -> its row of q / o and its query head.
struct RowAt {
    int token, head;
};
__device__ __forceinline__ RowAt row_at(const Params& p, const Item& it, int r) {
    const int t = r / p.group;
    return {it.r.row0 + it.tile * p.tokens_per_tile + t, it.head * p.group + (r - t * p.group)};
}

// The CTAs whose parts make up a split tile.
struct Parts {
    int first, last;
};
__device__ __forceinline__ Parts parts_of(const Params& p, const Item& it, const Start& st) {
    return {cta_of(st, it.tile_unit + p.item_cost), cta_of(st, it.tile_unit + it.cost - p.item_slack - 1)};
}
// Threads with ids 0 .. n-1 and their barrier `sync`: counts this CTA, whose part is stored; true in
// all of them if it was the last of `of` (`flag`: a shared int).
template <typename Sync>
__device__ bool last_of(uint32_t* counter, int of, int tid, int* flag, Sync sync) {
    sync();  // the CTA's stores come before thread 0's count, which releases them
    if (tid == 0) {
        uint32_t seen;  // and acquires those of the CTAs that counted before
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                     : "=r"(seen)
                     : "l"(static_cast<uint64_t>(__cvta_generic_to_global(counter)))
                     : "memory");
        *flag = seen == (uint32_t)(of - 1);
        if (*flag) *counter = 0;
    }
    sync();
    return *flag;
}
__device__ __forceinline__ int part_slot(const Parts& parts, int c) { return c == parts.first ? 0 : 1; }

// Tensor map of a pool for boxes of up to kKeyTile tokens of one head: (d, token, head, page).
bool make_pool_map(CUtensorMap* m, const moe_kv_cache& c, const void* base);

// attn_rows.cuh: requests of up to kFewRows rows a key/value head, on mma.sync, a tile's keys shared by
// warps; the second form is that for trees of drafted tokens (Params::tree)
cudaError_t launch_rows(const moe_kv_cache& c, Params& p, int rows, int grid_cap, cudaStream_t st);
cudaError_t launch_rows_tree(const moe_kv_cache& c, Params& p, int rows, int grid_cap, cudaStream_t st);
// attn_tile.cuh: query tiles of up to 256 rows on tcgen05; likewise
cudaError_t launch_tiles(const moe_kv_cache& c, Params& p, int grid_cap, cudaStream_t st);
cudaError_t launch_tiles_tree(const moe_kv_cache& c, Params& p, int grid_cap, cudaStream_t st);

inline int64_t most_units(const Params& p) {
    return ((int64_t)p.T / p.tokens_per_tile + p.B) * p.heads * ((int64_t)p.max_kv / kKeyTile + 2 + p.item_cost);
}
// One CTA per SM, and no more CTAs than there can be units.
inline int grid_for(const Params& p, int grid_cap) {
    int grid = device_info().num_sms;
    if (grid > grid_cap) grid = grid_cap;
    const int64_t units = most_units(p);
    return units < grid ? (int)units : grid;
}

}  // namespace attn
}  // namespace moe
