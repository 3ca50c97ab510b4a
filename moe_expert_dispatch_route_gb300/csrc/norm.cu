// moe_block_norm: what stands between two blocks, in one pass over their rows.
//   x = N(y; post) or y,   r' = resid + scale * gate * x,   out = N(r'; pre)
// Every row is read once and kept in registers as fp32 through both norms, so HBM bounds it: y and the
// residual in, both out.  A row is shared by kWarps warps, a thread holding kChunks times 8 consecutive
// elements; a norm is one sum over them and one exchange through shared memory.  A CTA of 256 threads (512
// for wide rows) takes as many rows as it has warps for, so that narrow rows fill it too.
// 16384 rows of 7168, bf16 with an fp32 residual, both norms and a gate, 1.41 GB: 234 us (6.0 TB/s; a copy of as many
// bytes reaches 6.8); 64 rows of 2048 2.2 us.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Rows of up to 4096 elements a CTA, 256 threads; wider ones 512.
template <int kWarps>
constexpr int kCtaThreads = kWarps > 8 ? 512 : 256;

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
    unpack8(__ldg(reinterpret_cast<const uint4*>(p)), x);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                   pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
}
// Rows that are read and written by this call alone: read once, past the L1 cache (out may be y, and
// resid_out resid: a thread reads its elements before it writes them).
__device__ __forceinline__ void read8(const float* p, float (&x)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void read8(const __nv_bfloat16* p, float (&x)[8]) {
    unpack8(__ldcs(reinterpret_cast<const uint4*>(p)), x);
}

// 1 / sqrt(mean + eps) of a row whose squares' sum over this thread's elements is `part`.  Two buffers of
// warps' sums, taken in turn, so that one barrier a norm is enough.
template <int kWarps>
__device__ __forceinline__ float inv_rms(float part, float* sums, int warp, float inv_n, float eps) {
    part = warp_sum(part);
    if (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) sums[warp] = part;
        __syncthreads();
        part = 0.0f;
        const int first = warp / kWarps * kWarps;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) part += sums[first + i];
    }
    return 1.0f / sqrtf(part * inv_n + eps);
}

template <typename T, typename R, int kWarps, int kChunks>
__global__ void __launch_bounds__(kCtaThreads<kWarps>, kChunks <= 2 ? 3 : 1)
    block_norm_kernel(const __grid_constant__ moe_norm_args a) {
    constexpr int kThreads = kCtaThreads<kWarps>;
    __shared__ float sums[2][kThreads / 32];
    pdl_begin();
    constexpr int kRows = kThreads / 32 / kWarps, kLanes = 32 * kWarps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x % kLanes, H = a.hidden, chunks = H / 8;
    const T *post = static_cast<const T*>(a.post_weight), *pre = static_cast<const T*>(a.pre_weight);
    const float inv_n = 1.0f / (float)H;
    // every thread of the CTA runs the same trips (barriers below)
    for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < a.T; t0 += (int64_t)gridDim.x * kRows) {
        const int64_t t = t0 + warp / kWarps;
        const int n = t < a.T ? chunks : 0;  // of this row
        const T* y = static_cast<const T*>(a.y) + t * H;
        const R* resid = static_cast<const R*>(a.resid) + t * H;
        const T* gate = static_cast<const T*>(a.gate) + (a.gate_rows > 1 ? t * H : 0);
        float x[kChunks][8], r[kChunks][8];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = lane + i * kLanes;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = r[i][j] = 0.0f;
            if (c < n) {
                read8(y + c * 8, x[i]);
                if (a.resid) read8(resid + c * 8, r[i]);
            }
        }
        if (post) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(x[i][j], x[i][j], sum);
            const float f = inv_rms<kWarps>(sum, sums[0], warp, inv_n, a.eps);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int c = lane + i * kLanes;
                if (c >= n) continue;
                float w[8];
                load8(post + c * 8, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = x[i][j] * f * w[j];
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = lane + i * kLanes;
            if (c >= n) continue;
            if (a.gate) {
                float g[8];
                load8(gate + c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] *= g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[i][j] = fmaf(a.scale, x[i][j], r[i][j]);
                sum = fmaf(r[i][j], r[i][j], sum);
            }
            if (a.resid_out) store8(static_cast<R*>(a.resid_out) + t * H + c * 8, r[i]);
        }
        if (a.out) {
            const float f = inv_rms<kWarps>(sum, sums[1], warp, inv_n, a.eps);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int c = lane + i * kLanes;
                if (c >= n) continue;
                float w[8];
                load8(pre + c * 8, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * f * w[j];
                store8(static_cast<T*>(a.out) + t * H + c * 8, r[i]);
            }
        }
        // a buffer is written again a whole row later: with one norm only, that takes a barrier
        if (kWarps > 1 && !(post && a.out)) __syncthreads();
    }
}

template <typename T, typename R, int kWarps, int kChunks>
cudaError_t launch_as(const moe_norm_args& a, int grid_cap, cudaStream_t st) {
    constexpr int kThreads = kCtaThreads<kWarps>, kRows = kThreads / 32 / kWarps;
    int grid = (a.T - 1) / kRows + 1;
    if (grid > grid_cap) grid = grid_cap;
    return launch_pdl(block_norm_kernel<T, R, kWarps, kChunks>, grid, kThreads, 0, st, a);
}
// A row goes to as few warps as hold it with 8 elements a thread, wide ones to 8 or 16 warps with more.  Three CTAs
// an SM keep enough loads under way: the rows above with 8 warps and 32 elements a thread take 242 us, 299 where the
// registers leave two CTAs; 32 warps 264.
template <typename T, typename R>
cudaError_t launch_of(const moe_norm_args& a, int grid_cap, cudaStream_t st) {
    const int n = (a.hidden / 8 + 31) / 32;  // warps' worth of chunks
    if (n <= 1) return launch_as<T, R, 1, 1>(a, grid_cap, st);
    if (n <= 2) return launch_as<T, R, 2, 1>(a, grid_cap, st);
    if (n <= 4) return launch_as<T, R, 4, 1>(a, grid_cap, st);
    if (n <= 8) return launch_as<T, R, 8, 1>(a, grid_cap, st);
    if (n <= 16) return launch_as<T, R, 8, 2>(a, grid_cap, st);
    if (n <= 32) return launch_as<T, R, 16, 2>(a, grid_cap, st);
    return launch_as<T, R, 16, 4>(a, grid_cap, st);
}

}  // namespace

cudaError_t launch_block_norm(const moe_norm_args& a, int grid_cap, cudaStream_t st) {
    const bool f = a.dtype == MOE_F32, rf = a.resid_dtype == MOE_F32;
    if (f) return rf ? launch_of<float, float>(a, grid_cap, st) : launch_of<float, __nv_bfloat16>(a, grid_cap, st);
    return rf ? launch_of<__nv_bfloat16, float>(a, grid_cap, st)
              : launch_of<__nv_bfloat16, __nv_bfloat16>(a, grid_cap, st);
}

}  // namespace moe
