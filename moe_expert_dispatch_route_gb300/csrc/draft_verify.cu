// moe_draft_verify: acceptance of drafted tokens and the draw of the one after them.
//
// The draw inverts a cumulative sum over the vocabulary.  Its terms are whole numbers (units
// of 2^-40), so partial sums may be formed in any order and split over any number of threads,
// and the token is the same: a thread-block cluster shares one request's row, each warp sums
// a contiguous segment, the 8 CTAs exchange their totals over distributed shared memory, and
// the CTA whose part holds the threshold reads the one warp's segment again (it is in L2), a few
// elements a thread.
// A large batch reads one row of the target a request, two where a token was refused, once; what bounds it is the
// latency of the loads under way and of each cluster's steps, not HBM: 256 requests of 131072 probabilities
// take 40.8 us in fp32 (4.8 TB/s) and 37.4 in bf16, half the bytes.  A single request is bound by the
// latency of the few dependent steps.  Eight small CTAs an SM let some clusters stream while others wait for
// their steps: with four CTAs of 256 threads fp32 takes 45 us, with two of 512 65.
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;  // CTAs sharing one request's row (the portable cluster size)
constexpr int kSegs = kCluster * kWarps;

struct VerifyParams {
    int V, max_draft;
    int most;  // drafted tokens a request may have: max_draft, or 0 where there are no ids
    int N;     // rows of drafted tokens that there are
    const void* target;
    int64_t target_ld;
    const void* draft;  // or null: q is 1 at the drafted token
    int64_t draft_ld;
    const int32_t* cu;
    const int32_t* ids;
    const float* u;
    const float* u_draw;
    int32_t* out_ids;
    int32_t* out_len;
    int32_t* err;
};

template <bool kF32>
__device__ __forceinline__ float prob(const void* base, int64_t i) {
    return kF32 ? static_cast<const float*>(base)[i] : bf16_bits_to_f(static_cast<const uint16_t*>(base)[i]);
}

// floor(2^40 * min(max(r, 0), 1)) in two 20-bit halves: adding 8 with rounding toward zero
// leaves floor(2^20 r) in the low bits of the sum; what is left of r is exact.
__device__ __forceinline__ void fixed40(float r, uint32_t& hi, uint32_t& lo) {
    r = fminf(fmaxf(r, 0.0f), 1.0f);  // NaN: 0
    const float a = __fadd_rz(r, 8.0f);
    const float b = __fadd_rz((r - (a - 8.0f)) * 0x1p20f, 8.0f);
    hi = __float_as_uint(a) - 0x41000000u;
    lo = __float_as_uint(b) - 0x41000000u;
}

// kVec consecutive values from element i (a multiple of kVec): 16 bytes, or one value.
template <bool kF32, int kVec>
__device__ __forceinline__ void load_vec(const void* row, int i, float (&x)[kVec]) {
    if (kVec == 1) {
        x[0] = prob<kF32>(row, i);
    } else if (kF32) {
        const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
        x[0] = f.x, x[1 % kVec] = f.y, x[2 % kVec] = f.z, x[3 % kVec] = f.w;
    } else {
        const uint4 f = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
        const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = bf16_bits_to_f((uint16_t)(w[e / 2 % 4] >> (16 * (e & 1))));
    }
}

// The weights of elements i .. i+kVec-1 (those below end).
template <bool kF32, int kVec>
struct Row {
    const void* p;
    const void* q;  // null: none
    int one;        // the token that a deterministic draft gave all its mass, -1: none

    __device__ __forceinline__ void load(int i, int end, float (&a)[kVec], float (&b)[kVec]) const {
#pragma unroll
        for (int e = 0; e < kVec; ++e) a[e] = b[e] = 0.0f;
        if (i >= end) return;  // segments end on multiples of kVec
        load_vec<kF32, kVec>(p, i, a);
        if (q) load_vec<kF32, kVec>(q, i, b);
    }
    __device__ __forceinline__ uint64_t weight(int i, float a, float b) const {
        if (i == one) b = 1.0f;
        uint32_t hi, lo;
        fixed40(a - b, hi, lo);
        return ((uint64_t)hi << 20) + lo;
    }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// This warp's sum over elements [lo, hi); the same in every lane.
template <bool kF32, int kVec>
__device__ uint64_t segment_sum(const Row<kF32, kVec>& row, int lo, int hi) {
    constexpr int kUnroll = kVec == 1 ? 16 : 16 / kVec;
    const int lane = threadIdx.x & 31;
    uint64_t sum = 0;
    for (int i0 = lo + lane * kVec; i0 < hi; i0 += 32 * kVec * kUnroll) {
        float a[kUnroll][kVec], b[kUnroll][kVec];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) row.load(i0 + u * 32 * kVec, hi, a[u], b[u]);
        uint32_t his = 0, los = 0;  // at most 16 * 2^20 each: no overflow
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                uint32_t h, l;
                if (i0 + u * 32 * kVec + e == row.one) b[u][e] = 1.0f;
                fixed40(a[u][e] - b[u][e], h, l);
                his += h;
                los += l;
            }
        sum += ((uint64_t)his << 20) + los;
    }
    return warp_sum64(sum);
}

// Whole CTA: the lowest element of [lo, hi) whose cumulative sum within the segment exceeds `want`
// (there is one), in the thread that finds it; -1 in the others.
template <bool kF32, int kVec>
__device__ int segment_find(const Row<kF32, kVec>& row, int lo, int hi, uint64_t want, uint64_t* warp_sums) {
    constexpr int kPer = 8, kLoads = kPer / kVec;  // consecutive elements of a thread
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i0 = lo; i0 < hi; i0 += kThreads * kPer) {
        const int i = i0 + threadIdx.x * kPer;
        float a[kLoads][kVec], b[kLoads][kVec];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) row.load(i + u * kVec, hi, a[u], b[u]);
        uint64_t w[kPer], mine = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            w[e] = i + e < hi ? row.weight(i + e, a[e / kVec][e % kVec], b[e / kVec][e % kVec]) : 0;
            mine += w[e];
        }
        uint64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        uint64_t run = incl - mine, all = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (k < warp) run += warp_sums[k];
            all += warp_sums[k];
        }
        __syncthreads();
        if (want < all) {  // the same in every thread
            if (want < run || want >= run + mine) return -1;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                run += w[e];
                if (want < run) return i + e;
            }
        }
        want -= all;
    }
    return -1;
}

template <bool kF32, int kVec>
__global__ void __launch_bounds__(kThreads, 8) __cluster_dims__(kCluster, 1, 1)
    draft_verify_kernel(const __grid_constant__ VerifyParams p, int B) {
    __shared__ uint64_t warp_tot[kWarps], find_sums[kWarps];
    __shared__ uint64_t cta_tot[2][kCluster];  // [pass][rank]: every CTA's total, written by its owner
    __shared__ int count_s;
    tc::cluster_sync();  // every CTA of the cluster runs before any writes another's shared memory
    pdl_begin();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank();
    // segments are whole vectors, equal but for the last ones
    const int vecs = (p.V + kVec - 1) / kVec;
    const int seg = (vecs + kSegs - 1) / kSegs * kVec;
    const int s0 = min((int)(rank * kWarps + warp) * seg, p.V), s1 = min(s0 + seg, p.V);
    // every CTA of a cluster walks the same requests: the cluster barriers below pair up
    for (int b = blockIdx.x / kCluster; b < B; b += gridDim.x / kCluster) {
        const int first = p.cu[b], n = p.cu[b + 1] - first;
        const bool ok = first >= 0 && n >= 0 && n <= p.most && first <= p.N - n;
        if (warp == 0) {  // how many drafted tokens are kept, and whether an id is out of range
            int c = 0, bad = 0;
            for (int i0 = 0; ok && i0 < n; i0 += 32) {
                bool kept = false;
                if (i0 + lane < n) {
                    const int i = i0 + lane, x = p.ids[first + i];
                    if (x < 0 || x >= p.V) {
                        bad = 1;
                    } else {
                        const float u = fminf(fmaxf(p.u[first + i], 0.0f), 1.0f - 0x1p-24f);
                        const float q = p.draft ? prob<kF32>(p.draft, (first + i) * p.draft_ld + x) : 1.0f;
                        const float t = prob<kF32>(p.target, ((int64_t)first + b + i) * p.target_ld + x);
                        // 24-bit significands: the product is exact in 64 bits
                        kept = (double)u * (double)q < (double)t;
                    }
                }
                const uint32_t m = __ballot_sync(0xffffffffu, kept);
                c += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
                if (m != 0xffffffffu) break;
            }
            if (bad) set_err(p.err, MOE_ERR_BAD_INDEX);
            if (lane == 0) count_s = c;
        }
        if (!ok) {
            if (rank == 0) {
                if (threadIdx.x == 0) {
                    set_err(p.err, MOE_ERR_BAD_INDEX);
                    p.out_len[b] = 0;
                }
                for (int i = threadIdx.x; i <= p.max_draft; i += kThreads)
                    p.out_ids[(int64_t)b * (p.max_draft + 1) + i] = -1;
            }
            continue;  // the same in every CTA of the cluster
        }
        __syncthreads();
        const int c = count_s;
        constexpr int kEl = kF32 ? 4 : 2;
        Row<kF32, kVec> row;
        row.p = static_cast<const uint8_t*>(p.target) + ((int64_t)first + b + c) * p.target_ld * kEl;
        row.q = p.draft && c < n ? static_cast<const uint8_t*>(p.draft) + ((int64_t)first + c) * p.draft_ld * kEl
                                 : nullptr;
        row.one = !p.draft && c < n ? p.ids[first + c] : -1;
        uint64_t total = 0, before = 0, own = 0;
        int pass = 0;
        for (;; ++pass) {
            const uint64_t s = segment_sum(row, s0, s1);
            if (lane == 0) warp_tot[warp] = s;
            __syncthreads();
            if (warp == 0) {
                const uint64_t t = warp_sum64(lane < kWarps ? warp_tot[lane] : 0);
                if (lane < kCluster) {
                    const uint32_t to = tc::map_to_rank(&cta_tot[pass][rank], (uint32_t)lane);
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(t) : "memory");
                }
            }
            tc::cluster_sync();
            total = before = 0;
            for (int r = 0; r < kCluster; ++r) {
                if (r < (int)rank) before += cta_tot[pass][r];
                total += cta_tot[pass][r];
            }
            own = cta_tot[pass][rank];
            if (total != 0 || pass == 1) break;
            row.q = nullptr;  // no mass beyond the draft's: draw from the target itself
            row.one = -1;
        }
        const float u = fminf(fmaxf(p.u_draw[b], 0.0f), 1.0f - 0x1p-24f);
        const uint64_t m = (uint64_t)(u * 0x1p24f);
        const uint64_t want = __umul64hi(m << 40, total);  // floor(m * total / 2^24)
        int32_t* out = p.out_ids + (int64_t)b * (p.max_draft + 1);
        if (want >= before && want < before + own) {  // this CTA's part holds the token
            uint64_t w = want - before;
            int seg_of = 0;
            for (; seg_of < kWarps - 1 && w >= warp_tot[seg_of]; ++seg_of) w -= warp_tot[seg_of];
            const int lo = min((int)(rank * kWarps + seg_of) * seg, p.V), hi = min(lo + seg, p.V);
            const int tok = segment_find(row, lo, hi, w, find_sums);
            if (tok >= 0) out[c] = tok;
        }
        if (rank == 0) {
            if (threadIdx.x == 0) {
                p.out_len[b] = c + 1;
                if (total == 0) {
                    out[c] = -1;
                    set_err(p.err, MOE_ERR_BAD_INDEX);
                }
            }
            for (int i = threadIdx.x; i <= p.max_draft; i += kThreads)
                if (i != c) out[i] = i < c ? p.ids[first + i] : -1;
        }
        // the next request writes cta_tot, warp_tot and count_s again
        tc::cluster_sync();
    }
}

}  // namespace

cudaError_t launch_draft_verify(int B, int N, int V, int max_draft, bool f32, const void* target, int64_t target_ld,
                                const void* draft, int64_t draft_ld, const int32_t* cu, const int32_t* ids,
                                const float* u, const float* u_draw, int32_t* out_ids, int32_t* out_len, int32_t* err,
                                int grid_cap, cudaStream_t st) {
    VerifyParams p{V,  max_draft, ids && u ? max_draft : 0, N, target, target_ld, draft, draft_ld, cu, ids, u, u_draw,
                   out_ids, out_len, err};
    // 16 bytes a load where every row starts on such a boundary and ends on one
    const int64_t lds = target_ld | (draft ? draft_ld : 0) | V;
    const bool vec = lds % (f32 ? 4 : 8) == 0 && aligned16(target) && aligned16(draft);
    int64_t clusters = grid_cap / kCluster < 1 ? 1 : grid_cap / kCluster;
    if (clusters > B) clusters = B;
    auto kern = f32 ? (vec ? draft_verify_kernel<true, 4> : draft_verify_kernel<true, 1>)
                    : (vec ? draft_verify_kernel<false, 8> : draft_verify_kernel<false, 1>);
    return launch_pdl(kern, (int)clusters * kCluster, kThreads, 0, st, p, B);
}

}  // namespace moe
