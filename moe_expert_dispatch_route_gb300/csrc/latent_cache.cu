// moe_latent_write: new tokens' latent vectors, normed on the way, and rotary keys into the pages of
// a cache.  HBM bounds it: 1152 bytes a token in and out (16384 tokens, 38 MB, 8.7 us, 4.3 TB/s with the launch; 64 tokens
// 2.0 us).  A warp takes a token: two pieces of 16 bytes of
// the latent vector a lane, one of the rotary key in the first 8, so the norm is one sum over the warp.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float square_sum(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
        s = fmaf(lo, lo, fmaf(hi, hi, s));
    }
    return s;
}
__device__ __forceinline__ uint4 scaled(uint4 v, uint4 weight, float f) {
    const uint32_t a[4] = {v.x, v.y, v.z, v.w}, b[4] = {weight.x, weight.y, weight.z, weight.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = pack_bf16x2(__uint_as_float(a[j] << 16) * f * __uint_as_float(b[j] << 16),
                           __uint_as_float(a[j] & 0xffff0000u) * f * __uint_as_float(b[j] & 0xffff0000u));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool kNorm>
__global__ void __launch_bounds__(kThreads) latent_write_kernel(const __grid_constant__ moe_latent_cache c, int T,
                                                                const uint16_t* __restrict__ latent, int64_t ld_c,
                                                                const uint16_t* __restrict__ rope, int64_t ld_rope,
                                                                const uint16_t* __restrict__ weight, float eps,
                                                                const int64_t* __restrict__ slots, int32_t* err) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int64_t pool = (int64_t)c.num_pages * c.page_size;
    const int shift = __ffs(c.page_size) - 1;
    uint4 w[2];
    if (kNorm) {
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(weight) + lane + 32 * i);
    }
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < T; t += warps) {
        const int64_t slot = __ldg(slots + t);
        uint4 x[2], r = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = __ldcs(reinterpret_cast<const uint4*>(latent + t * ld_c) + lane + 32 * i);
        if (lane < 8) r = __ldcs(reinterpret_cast<const uint4*>(rope + t * ld_rope) + lane);
        if (slot < 0) continue;  // the whole warp
        if (slot >= pool) {
            if (lane == 0) set_err(err, MOE_ERR_BAD_INDEX);
            continue;
        }
        if (kNorm) {
            const float sum = warp_sum(square_sum(x[0]) + square_sum(x[1]));
            const float f = 1.0f / sqrtf(sum * (1.0f / 512.0f) + eps);
#pragma unroll
            for (int i = 0; i < 2; ++i) x[i] = scaled(x[i], w[i], f);
        }
        uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.kv) + (slot >> shift) * c.stride_page +
                                             (slot & (c.page_size - 1)) * c.stride_token);
#pragma unroll
        for (int i = 0; i < 2; ++i) to[lane + 32 * i] = x[i];
        if (lane < 8) to[64 + lane] = r;
    }
}

}  // namespace

cudaError_t launch_latent_write(const moe_latent_cache& c, int T, const void* latent, int64_t ld_c, const void* rope,
                                int64_t ld_rope, const void* weight, float eps, const int64_t* slots, int32_t* err,
                                int grid_cap, cudaStream_t st) {
    int grid = (T - 1) / (kThreads / 32) + 1;
    if (grid > grid_cap) grid = grid_cap;
    return launch_pdl(weight ? latent_write_kernel<true> : latent_write_kernel<false>, grid, kThreads, 0, st, c, T,
                      static_cast<const uint16_t*>(latent), ld_c, static_cast<const uint16_t*>(rope), ld_rope,
                      static_cast<const uint16_t*>(weight), eps, slots, err);
}

}  // namespace moe
