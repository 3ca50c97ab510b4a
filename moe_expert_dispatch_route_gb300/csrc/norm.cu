// moe_block_norm: what stands between two blocks, in one pass over their rows.
//   x = N(y; post) or y,   r' = resid + scale * gate * x,   out = N(r'; pre)
// Every row is read from HBM once and taken through both norms in fp32, so HBM bounds it: y and the residual in,
// both out.  A row is shared by kWarps warps, a thread holding kChunks times 8 consecutive elements; a norm is one
// sum over them and one exchange through shared memory.  Two kernels with the same arithmetic and order of sums (a
// row's result never depends on how many there are): CTAs that stay, with rows copied ahead, and, for narrow rows
// and those of which two do not fit an SM, plain loads into registers.
// 16384 rows of 7168, bf16 with an fp32 residual, both norms and a gate, 1.41 GB: 213 us (6.6 TB/s; 234 with plain
// loads); bf16 throughout 146 (188); 16384 of 4096 82 (128); 4096 of 16384 86 (166); 64 rows of 2048 2.5 us.
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

// Narrow rows share CTAs of 256 threads; one that is too wide for the ring has 512.
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
        const float* of = sums + warp / kWarps * kWarps;
        if (kWarps % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWarps; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(of + i);
                part += (v.x + v.y) + (v.z + v.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWarps; ++i) part += of[i];
        }
    }
    return rsqrtf(part * inv_n + eps);
}

template <typename T, typename R, int kWarps, int kChunks>
__global__ void __launch_bounds__(kCtaThreads<kWarps>, kChunks <= 2 ? 3 : 1)
    block_norm_kernel(const __grid_constant__ moe_norm_args a) {
    constexpr int kThreads = kCtaThreads<kWarps>;
    __shared__ __align__(16) float sums[2][kThreads / 32];
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

// CTAs that stay take the rows in turn.  The rows to come are copied into shared memory while one is normed, so
// the reads of HBM never wait for a norm's two exchanges, and a thread keeps its elements' weights in registers, as
// they are stored, from the first row on (loaded again for each row, 28 KB for 14 of y, they come from L2: 167 us
// where 146 are reached).  The row itself is read from shared memory twice: held in registers it spills (215).
constexpr int kMostStages = 8;
constexpr int kRingBytes = 208 * 1024;  // of an SM's CTAs together
struct StreamParams {
    moe_norm_args a;
    int stages, stage_bytes;  // a stage: one row of y, residual and gate
    int64_t inject_ns;
};
__device__ int32_t g_norm_error;  // read by moe_comm_error: MOE_ERR_TIMEOUT once a wait has run out
template <typename T>
struct Packed8;  // 8 elements as they are stored
template <>
struct Packed8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void shared(const float* p) {
        a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void to(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};
template <>
struct Packed8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void shared(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void to(float (&x)[8]) const { unpack8(v, x); }
};
// A CTA whose wait for its row-th row ran out: no row is copied any more, those under way land (or a bounded wait
// gives up) before the CTA ends, and its rows from that one on are void: NaN.
template <typename T, typename R, int kLanes>
__device__ __noinline__ void leave(const StreamParams& sp, uint64_t* full, uint64_t* never, int row) {
    const moe_norm_args& a = sp.a;
    const int64_t first = blockIdx.x + (int64_t)row * gridDim.x;
    if (threadIdx.x == 0) {
        if (sp.inject_ns > 0) tc::wait_on_nothing(never, (uint64_t)sp.inject_ns);
        set_err(&g_norm_error, MOE_ERR_TIMEOUT);
        for (int i = 0; i < sp.stages && first + (int64_t)i * gridDim.x < a.T; ++i)
            tc::mbar_wait_bounded(&full[(row + i) % sp.stages], (row + i) / sp.stages & 1);
    }
    const float nan = __int_as_float(0x7fc00000);
    const float none[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
    for (int64_t t = first; t < a.T; t += gridDim.x)
        for (int c = threadIdx.x; c < a.hidden / 8; c += kLanes) {
            if (a.resid_out) store8(static_cast<R*>(a.resid_out) + t * a.hidden + c * 8, none);
            if (a.out) store8(static_cast<T*>(a.out) + t * a.hidden + c * 8, none);
        }
}
template <typename T, typename R, int kWarps, int kChunks, int kCtas>
__global__ void __launch_bounds__(kWarps * 32, kCtas) block_norm_stream_kernel(const __grid_constant__ StreamParams sp) {
    constexpr int kLanes = 32 * kWarps;
    const moe_norm_args& a = sp.a;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) float sums[2][kWarps];
    __shared__ uint64_t full[kMostStages], never;
    __shared__ int gave_up;  // the CTA's row whose wait ran out first
    const int tid = threadIdx.x, warp = tid >> 5, H = a.hidden, chunks = H / 8;
    const int y_bytes = H * (int)sizeof(T), r_bytes = a.resid ? H * (int)sizeof(R) : 0;
    const bool gates = a.gate && a.gate_rows > 1;
    if (tid == 0) {
        for (int i = 0; i < sp.stages; ++i) tc::mbar_init(&full[i], 1);
        tc::mbar_init(&never, 1);
        gave_up = INT32_MAX;
        tc::fence_barrier_init();
    }
    __syncthreads();
    pdl_begin();
    auto fetch = [&](int64_t t, int st) {  // one thread
        if (t >= a.T) return;
        uint8_t* to = ring + st * sp.stage_bytes;
        tc::mbar_arrive_expect_tx(&full[st], sp.stage_bytes);
        tc::bulk_load(to, static_cast<const T*>(a.y) + t * H, y_bytes, &full[st]);
        if (r_bytes) tc::bulk_load(to + y_bytes, static_cast<const R*>(a.resid) + t * H, r_bytes, &full[st]);
        if (gates) tc::bulk_load(to + y_bytes + r_bytes, static_cast<const T*>(a.gate) + t * H, y_bytes, &full[st]);
    };
    if (tid == 0)
        for (int i = 0; i < sp.stages; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
    const T *post = static_cast<const T*>(a.post_weight), *pre = static_cast<const T*>(a.pre_weight);
    Packed8<T> wp[kChunks], wn[kChunks], g[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = tid + i * kLanes;
        if (c >= chunks) continue;
        if (post) wp[i].load(post + c * 8);
        if (a.out) wn[i].load(pre + c * 8);
        if (a.gate && !gates) g[i].load(static_cast<const T*>(a.gate) + c * 8);
    }
    const float inv_n = 1.0f / (float)H;
    volatile int* left = &gave_up;
    const bool hook = sp.inject_ns > 0 && blockIdx.x == 0;  // test hook: as if the first row's wait had run out
    int st = 0, turn = 0, row = 0;
    uint32_t parity = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, ++row) {
        const bool landed = tc::mbar_wait_bounded(&full[st], parity) && !hook;
        if (!landed) atomicMin(&gave_up, row);
        const uint8_t* at = ring + st * sp.stage_bytes;
        const T *y = reinterpret_cast<const T*>(at), *gate = reinterpret_cast<const T*>(at + y_bytes + r_bytes);
        const R* resid = reinterpret_cast<const R*>(at + y_bytes);
        const float start = landed ? 0.0f : __int_as_float(0x7fc00000);  // of a sum: a wait that gave up makes it NaN
        float f = 1.0f, sum = start;
        if (post) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int c = tid + i * kLanes;
                if (c >= chunks) continue;
                Packed8<T> y8;
                float x[8];
                y8.shared(y + c * 8);
                y8.to(x);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
            }
            f = inv_rms<kWarps>(sum, sums[turn], warp, inv_n, a.eps), turn ^= 1, sum = start;
        }
        float r[kChunks][8];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = tid + i * kLanes;
            if (c >= chunks) continue;
            Packed8<T> y8;
            float x[8], w[8];
            y8.shared(y + c * 8);
            y8.to(x);
            if (post) {
                wp[i].to(w);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * f * w[j];
            }
            if (a.gate) {
                if (gates) g[i].shared(gate + c * 8);
                g[i].to(w);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = 0.0f;
            if (r_bytes) {
                Packed8<R> r8;
                r8.shared(resid + c * 8);
                r8.to(r[i]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[i][j] = fmaf(a.scale, x[j], r[i][j]);
                sum = fmaf(r[i][j], r[i][j], sum);
            }
            if (a.resid_out) store8(static_cast<R*>(a.resid_out) + t * H + c * 8, r[i]);
        }
        if (a.out)
            f = inv_rms<kWarps>(sum, sums[turn], warp, inv_n, a.eps), turn ^= 1;
        else
            __syncthreads();
        // behind this barrier a wait of this row that ran out is known to all (by its number: a faster thread may tell of
        // the next row's already), through the norm's sum where there is one: reading the word for every row costs 3 %
        if ((!a.out || f != f) && *left <= row) break;
        // and every thread has read its numbers: the stage takes another row
        if (tid == 0) fetch(t + (int64_t)sp.stages * gridDim.x, st);
        if (++st == sp.stages) st = 0, parity ^= 1u;
        if (!a.out) continue;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = tid + i * kLanes;
            if (c >= chunks) continue;
            float w[8];
            wn[i].to(w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * f * w[j];
            store8(static_cast<T*>(a.out) + t * H + c * 8, r[i]);
        }
    }
    if (*left != INT32_MAX) leave<T, R, kLanes>(sp, full, &never, *left);
}

template <typename T, typename R, int kWarps, int kChunks>
cudaError_t launch_as(const moe_norm_args& a, int grid_cap, cudaStream_t st) {
    constexpr int kThreads = kCtaThreads<kWarps>, kRows = kThreads / 32 / kWarps;
    int grid = (a.T - 1) / kRows + 1;
    if (grid > grid_cap) grid = grid_cap;
    return launch_pdl(block_norm_kernel<T, R, kWarps, kChunks>, grid, kThreads, 0, st, a);
}
// How far ahead rows are copied: HBM needs some 45 KB an SM under way, and slows down to 86 % when reads press
// on the writes (32768 rows of 4096, one norm: 161 us with 32 KB ahead, 181 with 64; 16384 of 7168 with an fp32
// residual and a gate a token, two norms: 250 with 57 KB, 281 with 115; 16384 of 4096, two norms: 82 with 64, 86
// with 32).  Two norms take longer, so a little more of it waits.
template <typename T, typename R, int kWarps, int kChunks, int kCtas>
cudaError_t launch_stream(const moe_norm_args& a, int stage_bytes, int grid_cap, cudaStream_t st) {
    constexpr int kRing = kRingBytes / kCtas;
    auto kern = block_norm_stream_kernel<T, R, kWarps, kChunks, kCtas>;
    const cudaError_t e = ensure_max_dynamic_smem(kern, kRing);
    if (e != cudaSuccess) return e;
    const int ahead = (a.post_weight && a.out ? 48 : 40) * 1024 / kCtas;
    int stages = 1 + (ahead + stage_bytes / 2) / stage_bytes;
    if (stages < 2) stages = 2;
    if (stages > kMostStages) stages = kMostStages;
    if (stages > kRing / stage_bytes) stages = kRing / stage_bytes;
    int grid = device_info().num_sms * kCtas;
    if (grid > a.T) grid = a.T;
    if (grid > grid_cap) grid = grid_cap;
    return launch_pdl(kern, grid, kWarps * 32, stages * stage_bytes, st, StreamParams{a, stages, stage_bytes, wait_injection_ns()});
}
// Few warps a row keep a norm's exchange short, and a fitting count of chunks wastes few threads (fp32 weights take
// twice the registers: twice the warps there).  A row of 7168 takes its CTA some 1.9 us: with bf16 throughout two
// CTAs an SM hide one another's exchanges (146 us for 16384 rows, 202 with one; two of 16 warps 175, one of 32 204);
// wide rows with more bytes an element fill HBM with one, and two slow it down (fp32 residual: 213 against 239; 5120
// elements 154, 171; 4096 with a gate a token 140, 157; but of 4104, 25 KB, one takes 157 and two 132).  `one` says
// that: more than five bytes an element are an fp32 residual, a gate a token beside a residual, or fp32 rows with either.
template <typename T, typename R>
cudaError_t launch_of(const moe_norm_args& a, int grid_cap, cudaStream_t st) {
    const int n = (a.hidden / 8 + 31) / 32;  // warps' worth of chunks
    const int row = a.hidden * (int)(sizeof(T) + (a.resid ? sizeof(R) : 0) + (a.gate && a.gate_rows > 1 ? sizeof(T) : 0));
    constexpr bool kHalf = sizeof(T) == 2;
    const bool one = row > 28 * 1024 && row > 5 * a.hidden;
    if (n <= 1) return launch_as<T, R, 1, 1>(a, grid_cap, st);
    if (n <= 2) return launch_as<T, R, 2, 1>(a, grid_cap, st);
    // up to 1024 elements plain loads do as well until rows come in tens an SM (4096 rows of 1024: 7.7 us, staying
    // CTAs 8.3; 16384: 31 and 26)
    if (n <= 4 && a.T < 32 * device_info().num_sms) return launch_as<T, R, 4, 1>(a, grid_cap, st);
    if (n <= 4) return launch_stream<T, R, 4, 1, 8>(a, row, grid_cap, st);
    // up to 2048: a chunk a thread, four CTAs an SM (16384 rows of 2048, bf16: 45 us; two CTAs 57, plain loads 53, four
    // warps of two chunks 46; 4096 of 1536: 11.4, 15.8, 13.5, 12.2; of 2048 with an fp32 residual two CTAs would take
    // 64 of these 70, and 86 of 95 in fp32 throughout)
    if (n <= 8) return launch_stream<T, R, 8, 1, 4>(a, row, grid_cap, st);
    // a little above, three chunks a thread of four warps waste fewer threads than two of eight (16384 rows of 2560,
    // bf16: 53 us, 74; 4096: 16.5, 22.1; with an fp32 residual 85, 79 and 23.0, 22.5)
    if constexpr (kHalf)
        if (n <= 12) return launch_stream<T, R, 4, 3, 4>(a, row, grid_cap, st);
    if (n <= 16)
        return one ? launch_stream<T, R, 8, 2, 1>(a, row, grid_cap, st) : launch_stream<T, R, 8, 2, 2>(a, row, grid_cap, st);
    if constexpr (kHalf) {
        if (n <= 24)
            return one ? launch_stream<T, R, 8, 3, 1>(a, row, grid_cap, st)
                       : launch_stream<T, R, 8, 3, 2>(a, row, grid_cap, st);
        if (n <= 32)
            return one ? launch_stream<T, R, 8, 4, 1>(a, row, grid_cap, st)
                       : launch_stream<T, R, 8, 4, 2>(a, row, grid_cap, st);
        if (row <= kRingBytes / 2) return launch_stream<T, R, 16, 4, 1>(a, row, grid_cap, st);
    } else if (n <= 32) {
        return launch_stream<T, R, 16, 2, 1>(a, row, grid_cap, st);
    }
    return launch_as<T, R, 16, 4>(a, grid_cap, st);
}

}  // namespace

int32_t* norm_error_word() {
    void* p = nullptr;
    return cudaGetSymbolAddress(&p, g_norm_error) == cudaSuccess ? static_cast<int32_t*>(p) : nullptr;
}

cudaError_t launch_block_norm(const moe_norm_args& a, int grid_cap, cudaStream_t st) {
    const bool f = a.dtype == MOE_F32, rf = a.resid_dtype == MOE_F32;
    if (f) return rf ? launch_of<float, float>(a, grid_cap, st) : launch_of<float, __nv_bfloat16>(a, grid_cap, st);
    return rf ? launch_of<__nv_bfloat16, float>(a, grid_cap, st)
              : launch_of<__nv_bfloat16, __nv_bfloat16>(a, grid_cap, st);
}

}  // namespace moe
