// The paged key/value cache: moe_kv_write stores new tokens' keys and values (quantised to
// e4m3 for an FP8 cache), moe_kv_read brings cached tokens back to packed bf16 rows.
// Both only move bytes, so HBM bounds them; a thread moves 16 bytes of bf16 at a time.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -100, kMaxExp = 119;  // e4m3 codes times 2^s stay exact, finite bf16 values

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// ---------------------------------------------------------------- write
// kLanes = head_dim / 8 lanes hold one (token, k or v, head) row, 8 values each, and take the
// heads of a token in turn, kUnroll rows on their way at once: slot and addresses are found once a
// token.  A row's largest magnitude is a maximum over packed bf16 pairs and kLanes lanes.
// The e4m3 form is bound by issue slots before it is by HBM, so its scale comes from the bits of
// the largest bf16 magnitude and scaling is one product.
// 16384 tokens of 8 heads of 128 into e4m3, 101 MB, in random slots: 21.4 us (4.7 TB/s; 20.2 without
// the scales, which are single bytes); into bf16, 134 MB, 22.3 us (6.0 TB/s); 64 tokens of 4 bf16 heads 1.5 us.
constexpr int kUnroll = 4;

template <int kLanes, bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const __grid_constant__ moe_kv_cache c, int T,
                                                            const uint16_t* __restrict__ k,
                                                            const uint16_t* __restrict__ v, int64_t ld_k, int64_t ld_v,
                                                            int64_t head_stride, const int64_t* __restrict__ slots,
                                                            int32_t* err) {
    pdl_begin();
    const int lane = threadIdx.x % kLanes;
    const int H = c.num_heads;
    const int64_t pool = (int64_t)c.num_pages * c.page_size;
    const int shift = __ffs(c.page_size) - 1;
    // groups of kLanes lanes over (token, k or v, run of kUnroll heads); every lane of a warp runs
    // the same trips (shuffles below)
    const int runs = (H + kUnroll - 1) / kUnroll, items = T * 2 * runs;  // host: fits
    const int ngroups = gridDim.x * (kThreads / kLanes);
    const int mine = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;  // threads may be more than 2^32
    const int warp_first = blockIdx.x * (kThreads / kLanes) + (threadIdx.x & ~31) / kLanes;
    for (int i = mine, w0 = warp_first; w0 < items; i += ngroups, w0 += ngroups) {
        const int at = min(i, items - 1), h0 = at % runs * kUnroll, t = at / runs >> 1;
        const bool is_v = at / runs & 1;
        const uint16_t* src = (is_v ? v + t * ld_v : k + t * ld_k) + h0 * head_stride;
        uint4 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            x[u] = make_uint4(0, 0, 0, 0);
            if (h0 + u < H) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + u * head_stride) + lane);
        }
        const int64_t slot = i < items ? slots[t] : -1;
        if (slot >= pool && lane == 0) set_err(err, MOE_ERR_BAD_INDEX);
        const bool ok = slot >= 0 && slot < pool;
        const int64_t page = slot >> shift;
        const int tok = (int)slot & (c.page_size - 1);
        void* dst = is_v ? c.v : c.k;
        const int64_t to = page * c.stride_page + h0 * c.stride_head + tok * c.stride_token;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (h0 + u >= H) break;
            if (!kFp8) {
                if (ok) reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + to + u * c.stride_head)[lane] = x[u];
                continue;
            }
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t m = 0;  // the largest magnitude as bf16 bits: ordered as integers, NaN above infinity
#pragma unroll
            for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7fff7fffu);
            m = max(m & 0xffffu, m >> 16);
            // the lanes of a group alone: the other group of the warp may have fewer heads left
            const uint32_t group = kLanes == 32 ? 0xffffffffu
                                                : ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(group, m, o));
            if (!ok) continue;
            // 448 = 1.75 * 2^8: s is amax's exponent less 8, one more above a significand of 1.75; the
            // limits cover subnormals and infinity
            const int s = m == 0 ? 0 : min(max((int)(m >> 7) - 135 + ((m & 0x7f) > 0x60), kMinExp), kMaxExp);
            const float f = __int_as_float((127 - s) << 23);
            uint32_t q[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                q[j] = (uint32_t)f2_to_e4m3x2(bf_lo(w[2 * j]) * f, bf_hi(w[2 * j]) * f) |
                       ((uint32_t)f2_to_e4m3x2(bf_lo(w[2 * j + 1]) * f, bf_hi(w[2 * j + 1]) * f) << 16);
            reinterpret_cast<uint2*>(static_cast<uint8_t*>(dst) + to + u * c.stride_head)[lane] = make_uint2(q[0], q[1]);
            if (lane == 0)
                (is_v ? c.v_scale : c.k_scale)[(page * H + h0 + u) * c.page_size + tok] =
                    m > 0x7f80u ? 255 : (uint8_t)(s + 127);
        }
    }
}

// ---------------------------------------------------------------- read
// The 8 values of 8 e4m3 codes under 2^s: every step is exact for a scale moe_kv_write stores.
__device__ __forceinline__ uint4 dequant8(uint2 q, uint8_t b) {
    const float f = b == 255 ? __uint_as_float(0x7fc00000u) : b == 0 ? 0x1p-127f : __uint_as_float((uint32_t)b << 23);
    const uint32_t w[2] = {q.x, q.y};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2_raw two = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
        const float2 v = __half22float2(__half2(two));
        o[j] = pack_bf16x2(v.x * f, v.y * f);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A warp takes kRows consecutive output rows: lane i < kRows finds row i's request by
// bisection of cu_len and its page, then all lanes copy the rows' 2 * heads * kLanes pieces of
// 16 output bytes, kUnroll loads in flight each.
// 4 prefixes of up to 32768 e4m3 tokens, 8 heads of 128, 296 MB: 51.2 us (5.8 TB/s, four fifths of it
// writes); 13 bf16 prefixes of up to 700 3.2 us, a chain of three dependent loads.
constexpr int kRows = 4;

template <int kLanes, bool kFp8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ moe_kv_cache c, int B, int T,
                                                           const int32_t* __restrict__ table, int table_ld,
                                                           const int32_t* __restrict__ start,
                                                           const int32_t* __restrict__ cu, uint4* __restrict__ k_out,
                                                           uint4* __restrict__ v_out, int32_t* err) {
    pdl_begin();
    constexpr int kUnroll = 8;
    const int lane = threadIdx.x & 31;
    const int H = c.num_heads;
    const int pieces = 2 * H * kLanes;  // of one row
    const int shift = __ffs(c.page_size) - 1;
    const int total = min(T, cu[B]);
    const int warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), nwarps = gridDim.x * (kThreads / 32);
    for (int64_t first = (int64_t)warp * kRows; first < total; first += (int64_t)nwarps * kRows) {
        int64_t at = -1, sat = 0;  // lane i: element and scale offset of row i's head 0; -1: no such row
        if (lane < kRows && first + lane < total) {
            const int r = (int)first + lane;
            int lo = 0, hi = B;  // cu[lo] <= r < cu[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= r) lo = mid; else hi = mid;
            }
            const int64_t pos = (int64_t)start[lo] + (r - cu[lo]);
            const int64_t col = pos >> shift;
            int page = -1;
            if (pos >= 0 && col < table_ld) page = table[(int64_t)lo * table_ld + col];
            if (page < 0 || page >= c.num_pages) {
                set_err(err, MOE_ERR_BAD_INDEX);
            } else {
                const int tok = (int)pos & (c.page_size - 1);
                at = page * c.stride_page + tok * c.stride_token;
                sat = (int64_t)page * H * c.page_size + tok;
            }
        }
        int64_t ats[kRows], sats[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            ats[i] = __shfl_sync(0xffffffffu, at, i);
            sats[i] = __shfl_sync(0xffffffffu, sat, i);
        }
        for (int p0 = lane; p0 < pieces; p0 += 32 * (kUnroll / kRows)) {
            uint4 x[kUnroll];
            uint8_t sc[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = u % kRows, p = p0 + (u / kRows) * 32;
                x[u] = make_uint4(0, 0, 0, 0);
                sc[u] = 0;
                if (p < pieces && ats[i] >= 0) {
                    const int row = p / kLanes, part = p % kLanes;
                    const bool is_v = row >= H;
                    const int h = is_v ? row - H : row;
                    const int64_t e = ats[i] + h * c.stride_head;
                    if (kFp8) {
                        const uint2 q = __ldcs(
                            reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? c.v : c.k) + e) + part);
                        x[u].x = q.x;
                        x[u].y = q.y;
                        sc[u] = (is_v ? c.v_scale : c.k_scale)[sats[i] + (int64_t)h * c.page_size];
                    } else {
                        x[u] = __ldcs(
                            reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(is_v ? c.v : c.k) + e) + part);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = u % kRows, p = p0 + (u / kRows) * 32;
                if (p < pieces && ats[i] >= 0) {
                    const int row = p / kLanes;
                    const bool is_v = row >= H;
                    const int64_t o = ((first + i) * H + (is_v ? row - H : row)) * kLanes + p % kLanes;
                    __stcs((is_v ? v_out : k_out) + o, kFp8 ? dequant8(make_uint2(x[u].x, x[u].y), sc[u]) : x[u]);
                }
            }
        }
    }
}

template <int kLanes, bool kFp8>
cudaError_t write_as(const moe_kv_cache& c, int T, const void* k, const void* v, int64_t ld_k, int64_t ld_v,
                     int64_t head_stride, const int64_t* slots, int32_t* err, int grid_cap, cudaStream_t st) {
    const int64_t items = (int64_t)T * 2 * ((c.num_heads + kUnroll - 1) / kUnroll);
    int64_t grid = (items * kLanes + kThreads - 1) / kThreads;
    if (grid > grid_cap) grid = grid_cap;
    auto kern = kv_write_kernel<kLanes, kFp8>;
    return launch_pdl(kern, (int)grid, kThreads, 0, st, c, T, static_cast<const uint16_t*>(k),
                      static_cast<const uint16_t*>(v), ld_k, ld_v, head_stride, slots, err);
}

template <int kLanes, bool kFp8>
cudaError_t read_as(const moe_kv_cache& c, int B, int T, const int32_t* table, int table_ld, const int32_t* start,
                    const int32_t* cu, void* k_out, void* v_out, int32_t* err, int grid_cap, cudaStream_t st) {
    int64_t grid = ((int64_t)T + kRows * (kThreads / 32) - 1) / (kRows * (kThreads / 32));
    if (grid > grid_cap) grid = grid_cap;
    return launch_pdl(kv_read_kernel<kLanes, kFp8>, (int)grid, kThreads, 0, st, c, B, T, table, table_ld, start, cu,
                      static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), err);
}

}  // namespace

cudaError_t launch_kv_write(const moe_kv_cache& c, int T, const void* k, const void* v, int64_t ld_k, int64_t ld_v,
                            int64_t head_stride, const int64_t* slots, int32_t* err, int grid_cap, cudaStream_t st) {
    const bool fp8 = c.dtype == MOE_FP8_E4M3;
    auto f = c.head_dim == 128 ? (fp8 ? write_as<16, true> : write_as<16, false>)
                               : (fp8 ? write_as<8, true> : write_as<8, false>);
    return f(c, T, k, v, ld_k, ld_v, head_stride, slots, err, grid_cap, st);
}

cudaError_t launch_kv_read(const moe_kv_cache& c, int B, int T, const int32_t* table, int table_ld,
                           const int32_t* start, const int32_t* cu, void* k_out, void* v_out, int32_t* err,
                           int grid_cap, cudaStream_t st) {
    const bool fp8 = c.dtype == MOE_FP8_E4M3;
    auto f = c.head_dim == 128 ? (fp8 ? read_as<16, true> : read_as<16, false>)
                               : (fp8 ? read_as<8, true> : read_as<8, false>);
    return f(c, B, T, table, table_ld, start, cu, k_out, v_out, err, grid_cap, st);
}

}  // namespace moe
