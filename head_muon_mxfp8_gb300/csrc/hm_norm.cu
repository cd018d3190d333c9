// RMS norm with the residual's addition and an MXFP8 output, and its gradient.
//
//   h = round(x + res);  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd gamma
//   (q, s) = MXFP8(y)
//   dx = dres + rstd (t - xhat mean(t xhat)),  t = dy gamma, xhat = h rstd
//   dgamma = sum over rows of dy xhat
// Every statistic is fp32 and of the stored h, so the gradient, which has only
// the stored h, differentiates exactly the function the forward pass computed.
// Memory-bound; a row stays in registers between its reduction and its output,
// so every tensor is read and written once.  8192 x 5120 bf16 with residual: norm
// 46.1 us (6.4 TB/s, 0.94 of the measured copy rate), gradient 54.6 us (6.1 TB/s,
// dgamma's second launch included); in fp32 81.7 and 100.3 us (6.7 TB/s both).
// The norm and rotation of heads has its own notes below.
// Far from it are the gradient's fp32 forms whose registers spill: 8192 rows of 6656
// columns without a residual's gradient 183 us (3.6 TB/s), of 16384 558 us with it and
// 439 without (3.8 and 3.7 TB/s).
#include "hm_internal.h"
#include "hm_mx_device.cuh"
#include "hm_ops.h"
#include "hm_ptx.cuh"
#include "hm_vec.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

namespace hm {

namespace {

constexpr int kMaxRowThreads = 512;
constexpr int kWarpRows = 8;       // rows per CTA where a row is one warp's
constexpr int kWarpMaxD = 1024;
constexpr int kMaxGradStages = 16;
constexpr int kGradRing = 208 * 1024;  // bytes of rows in flight per SM; a stage is at most 3 x 64 KB

// 8 elements of a row
template <bool F32>
struct Vec8;
template <>
struct Vec8<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        a = __ldcs(p);
        b = __ldcs(p + 1);
    }
    __device__ __forceinline__ void lds(const uint8_t* row, int j) {
        a = reinterpret_cast<const float4*>(row)[2 * j];
        b = reinterpret_cast<const float4*>(row)[2 * j + 1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void put(void* base, int64_t at, const float (&v)[8]) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    // rounds v to the type, storing it if base is given
    static __device__ __forceinline__ void round(void* base, int64_t at, float (&v)[8]) {
        if (base) put(base, at, v);
    }
};
template <>
struct Vec8<false> {
    uint4 a;
    __device__ __forceinline__ void load(const void* base, int64_t at) {
        a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    }
    __device__ __forceinline__ void lds(const uint8_t* row, int j) { a = reinterpret_cast<const uint4*>(row)[j]; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void put(void* base, int64_t at, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack(v);
    }
    static __device__ __forceinline__ void round(void* base, int64_t at, float (&v)[8]) {
        Vec8 r;
        r.a = pack(v);
        if (base) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = r.a;
        r.get(v);
    }
};

// (Ordinary loads: gamma, rstd and the partials may come from the kernel right
// before, which still runs when these start.)
__device__ __forceinline__ void load_f8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sum over the warp, the same in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, the same in every thread: warp sums, then the same tree
// over them in every warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.f);
}

// 1 / sqrt(sum / d + eps), off by little more than its own rounding: the quotient's
// and the sum's remainders are carried along (a product's or a quotient's remainder
// is one fma), and one Newton step on 1/sqrt removes its error.  Four roundings
// in a row instead moved 1.5 times as many codes off their 64-bit values.
__device__ __forceinline__ float inv_root(float sum, float d, float eps) {
    const float q = sum / d;
    const float a = q + eps;
    if (!(a >= 0x1p-100f && a <= 0x1p100f)) return 1.0f / sqrtf(a);  // the step below would leave fp32
    const float big = fmaxf(q, eps), small = fminf(q, eps);
    const float low = (small - (a - big)) + fmaf(-q, d, sum) / d;  // sum / d + eps - a
    const float y = rsqrtf(a);
    const float t = a * y;
    const float e = fmaf(-t, y, 1.0f) - fmaf(fmaf(a, y, -t), y, low * y * y);  // 1 - (a + low) y^2
    return fmaf(0.5f * e, y, y);
}

// A row per CTA, or per warp (8 rows per CTA) where a row has at most 1024
// columns: its sum then needs no barrier (32768 x 256 bf16: 19.0 us with a CTA
// per row, 10.4 with a warp; x 1024: 41.6 and 37.7).  A thread owns V vectors of 8 columns,
// vector i * (threads of the row) + t.
template <bool F32, int V, bool WARP>
__global__ void __launch_bounds__(kMaxRowThreads) rmsnorm_kernel(const __grid_constant__ RmsArgs p) {
    __shared__ float red[16];
    wait_for_earlier_kernels();
    const int t = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const int nv = p.d >> 3;
    const int lane = threadIdx.x & 31;
    const int64_t col_tiles = (p.d + 127) >> 7;
    uint8_t* srow = p.s + (row >> 7) * col_tiles * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4;
    if (row >= p.rows) {  // padding of the last scale tiles
        for (int64_t j = t; j < col_tiles; j += threads) *reinterpret_cast<uint32_t*>(srow + j * 512) = 0u;
        return;
    }
    float h[V][8];
    float sq = 0.f;  // pairs first, so that no chain of additions is longer than V
    Vec8<F32> x[V], r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * threads + t;
        if (j < nv) {
            x[i].load(p.x, row * p.ldx + j * 8);
            if (p.res) r[i].load(p.res, row * p.ldh + j * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * threads + t;
        if (j < nv) {
            x[i].get(h[i]);
            if (p.res) {
                float rv[8];
                r[i].get(rv);
#pragma unroll
                for (int k = 0; k < 8; ++k) h[i][k] += rv[k];
            }
            Vec8<F32>::round(p.h, row * p.ldh + j * 8, h[i]);
            float p4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) p4[k] = fmaf(h[i][2 * k + 1], h[i][2 * k + 1], h[i][2 * k] * h[i][2 * k]);
            sq += (p4[0] + p4[1]) + (p4[2] + p4[3]);
        }
    }
    const float rstd = inv_root(WARP ? warp_sum(sq) : block_sum(sq, red), static_cast<float>(p.d), p.eps);
    if (t == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * threads + t;
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (j < nv) {
            float gm[8];
            load_f8(p.gamma + j * 8, gm);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = h[i][k] * rstd * gm[k];
        }
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(y[k]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (p.block == 128) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
        }
        const int byte = mx_scale_byte(amax);
        const float sc = mx_inv_of_byte(byte);
        if (j < nv) {
            const uint32_t lo = cvt_e4m3x2(y[0] * sc, y[1] * sc) | (static_cast<uint32_t>(cvt_e4m3x2(y[2] * sc, y[3] * sc)) << 16);
            const uint32_t hi = cvt_e4m3x2(y[4] * sc, y[5] * sc) | (static_cast<uint32_t>(cvt_e4m3x2(y[6] * sc, y[7] * sc)) << 16);
            __stcs(reinterpret_cast<uint2*>(p.q + row * p.d + j * 8), make_uint2(lo, hi));
        }
        // the four scales of 128 columns as one word: bytes from lanes 0, 4, 8, 12 of each half warp
        uint32_t word = j < nv ? static_cast<uint32_t>(byte) << (8 * ((lane >> 2) & 3)) : 0u;
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if ((lane & 15) == 0 && j < nv) *reinterpret_cast<uint32_t*>(srow + (j >> 4) * 512) = word;
    }
}

// Gradient: one or two CTAs per SM take rows round-robin; a thread owns the same columns
// of every row (V vectors of 8, vector i * blockDim + t) and keeps their part of
// dgamma in registers.  The rows of dy, h and dres come into a ring of `stages`
// rows in shared memory by bulk copies issued several rows ahead -- loading a row
// into registers only when its turn came left the memory idle during every
// reduction (3.6 TB/s at 8192 x 5120 bf16).  One barrier per row: it publishes
// the warps' sums of t xhat and says that the row has been read, so thread 0
// refills its stage right behind it.  Waits are bounded (HM_ERR_TIMEOUT).
template <bool F32>
__device__ __forceinline__ void fill_stage(const RmsGradArgs& p, uint8_t* stage, uint64_t* bar, int64_t row) {
    const uint32_t bytes = static_cast<uint32_t>(p.d) * (F32 ? 4 : 2);
    const int64_t es = F32 ? 4 : 2;
    mbar_arrive_expect_tx(smem_u32(bar), bytes * (p.dres ? 3 : 2));
    const uint32_t dst = smem_u32(stage);
    bulk_load(dst, static_cast<const char*>(p.dy) + row * p.lddy * es, bytes, smem_u32(bar));
    bulk_load(dst + bytes, static_cast<const char*>(p.h) + row * p.ldh * es, bytes, smem_u32(bar));
    if (p.dres) bulk_load(dst + 2 * bytes, static_cast<const char*>(p.dres) + row * p.ldh * es, bytes, smem_u32(bar));
}

// T: most threads, B: CTAs per SM.  gamma stays in registers where they suffice.
template <bool F32, int V, int T, int B>
__global__ void __launch_bounds__(T, B) rmsnorm_grad_kernel(const __grid_constant__ RmsGradArgs p) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][T / 32];
    __shared__ uint64_t full[kMaxGradStages];
    __shared__ int bail_word;
    volatile int* bail = &bail_word;
    const int nv = p.d >> 3;
    const int row_bytes = p.d * (F32 ? 4 : 2);
    const int stage_bytes = row_bytes * (p.dres ? 3 : 2);
    const int stages = p.stages;
    const int64_t mine = (p.rows - blockIdx.x + gridDim.x - 1) / gridDim.x;  // rows of this CTA
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full[s]), 1);
        bail_word = 0;
        fence_mbar_init();
    }
    __syncthreads();
    wait_for_earlier_kernels();
    if (threadIdx.x == 0 && !p.inject)
        for (int s = 0; s < stages && s < mine; ++s)
            fill_stage<F32>(p, ring + s * stage_bytes, &full[s], blockIdx.x + static_cast<int64_t>(s) * gridDim.x);
    constexpr bool kKeepGamma = V == 1 || T * B <= 640;
    float dg[V][8], gamma[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * blockDim.x + threadIdx.x;
        if (kKeepGamma && j < nv) load_f8(p.gamma + j * 8, gamma[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k) dg[i][k] = 0.f;
    }
    const float inv_d = 1.0f / static_cast<float>(p.d);
    int s = 0;
    uint32_t ph = 0;
    float rstd_next = mine > 0 ? p.rstd[blockIdx.x] : 0.f;
    int64_t it = 0;
    for (; it < mine; ++it) {
        const int64_t row = blockIdx.x + it * gridDim.x;
        const float rstd = rstd_next;
        if (it + 1 < mine) rstd_next = p.rstd[row + gridDim.x];
        const int ok = mbar_wait<false>(smem_u32(&full[s]), ph, p.err, bail);
        const uint8_t* stage = ring + s * stage_bytes;
        Vec8<F32> dy[V], h[V], dr[V];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = i * blockDim.x + threadIdx.x;
            if (j < nv) {
                dy[i].lds(stage, j);
                h[i].lds(stage + row_bytes, j);
                if (p.dres) dr[i].lds(stage + 2 * row_bytes, j);
                float y[8], x[8];
                if (!kKeepGamma) load_f8(p.gamma + j * 8, gamma[i]);
                dy[i].get(y);
                h[i].get(x);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float yx = y[k] * (x[k] * rstd);
                    dg[i][k] += yx;
                    dot = fmaf(yx, gamma[i][k], dot);
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if ((threadIdx.x & 31) == 0) red[it & 1][threadIdx.x >> 5] = dot;
        if (!__syncthreads_and(ok)) break;
        if (threadIdx.x == 0 && it + stages < mine)
            fill_stage<F32>(p, ring + s * stage_bytes, &full[s], row + static_cast<int64_t>(stages) * gridDim.x);
        if (++s == stages) { s = 0; ph ^= 1u; }
        // every warp adds the warps' sums the same way: lane k holds warp k's
        float mean = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[it & 1][threadIdx.x & 31] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
        const float back = -rstd * (mean * inv_d);  // dx = dres + rstd t - xhat rstd mean
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = i * blockDim.x + threadIdx.x;
            if (j < nv) {
                float y[8], x[8], o[8], rv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (!kKeepGamma) load_f8(p.gamma + j * 8, gamma[i]);
                dy[i].get(y);
                h[i].get(x);
                if (p.dres) dr[i].get(rv);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = fmaf(x[k] * rstd, back, fmaf(y[k] * gamma[i][k], rstd, rv[k]));
                Vec8<F32>::put(p.dx, row * p.ldh + j * 8, o);
            }
        }
    }
    // after a wait that gave up: this CTA's copies still in flight
    if (it < mine && threadIdx.x == 0 && !p.inject)
        for (int k = 0; k < stages; ++k) {
            const int64_t i = it + k;
            if (i >= mine) break;
            mbar_wait(smem_u32(&full[i % stages]), static_cast<uint32_t>(i / stages) & 1u, p.err, bail, false);
        }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * blockDim.x + threadIdx.x;
        if (j < nv) {
            float4* out = reinterpret_cast<float4*>(p.partials + static_cast<int64_t>(blockIdx.x) * p.d + j * 8);
            out[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
            out[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
        }
    }
}

// Gradient of rows of at most 1024 columns: a warp per row, no barrier until the
// end (32768 x 256 bf16: 73.6 us through the ring, 15.4; x 1024: 83.5 and 51.9), the
// next row's vectors loaded before this one's are used (V <= 2; more would not
// leave registers); the warps' parts of dgamma are added in order.
template <bool F32, int V>
__global__ void __launch_bounds__(32 * kWarpRows) rmsnorm_grad_warp_kernel(const __grid_constant__ RmsGradArgs p) {
    __shared__ __align__(16) float part[kWarpRows][V * 256];
    constexpr bool kAhead = V <= 2;
    wait_for_earlier_kernels();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nv = p.d >> 3;
    float dg[V][8], gamma[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j = i * 32 + lane;
#pragma unroll
        for (int k = 0; k < 8; ++k) dg[i][k] = gamma[i][k] = 0.f;
        if (kAhead && j < nv) load_f8(p.gamma + j * 8, gamma[i]);
    }
    Vec8<F32> dy[V], h[V], dr[V], dy1[V], h1[V], dr1[V];
    auto fetch = [&](int64_t row, Vec8<F32>(&a)[V], Vec8<F32>(&b)[V], Vec8<F32>(&c)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = i * 32 + lane;
            if (j < nv) {
                a[i].load(p.dy, row * p.lddy + j * 8);
                b[i].load(p.h, row * p.ldh + j * 8);
                if (p.dres) c[i].load(p.dres, row * p.ldh + j * 8);
            }
        }
    };
    const float inv_d = 1.0f / static_cast<float>(p.d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarpRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kWarpRows + warp;
    float rstd1 = 0.f;
    if (row < p.rows) {
        fetch(row, dy, h, dr);
        rstd1 = p.rstd[row];
    }
    for (; row < p.rows; row += step) {
        const float rstd = rstd1;
        const bool more = row + step < p.rows;
        if (more) {
            rstd1 = p.rstd[row + step];
            if (kAhead) fetch(row + step, dy1, h1, dr1);
        }
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = i * 32 + lane;
            if (j < nv) {
                float y[8], x[8];
                if (!kAhead) load_f8(p.gamma + j * 8, gamma[i]);
                dy[i].get(y);
                h[i].get(x);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float yx = y[k] * (x[k] * rstd);
                    dg[i][k] += yx;
                    dot = fmaf(yx, gamma[i][k], dot);
                }
            }
        }
        const float back = -rstd * (warp_sum(dot) * inv_d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = i * 32 + lane;
            if (j < nv) {
                float y[8], x[8], o[8], rv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (!kAhead) load_f8(p.gamma + j * 8, gamma[i]);
                dy[i].get(y);
                h[i].get(x);
                if (p.dres) dr[i].get(rv);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = fmaf(x[k] * rstd, back, fmaf(y[k] * gamma[i][k], rstd, rv[k]));
                Vec8<F32>::put(p.dx, row * p.ldh + j * 8, o);
            }
        }
        if (!more) break;
        if (kAhead) {
#pragma unroll
            for (int i = 0; i < V; ++i) dy[i] = dy1[i], h[i] = h1[i], dr[i] = dr1[i];
        } else {
            fetch(row + step, dy, h, dr);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float4* q = reinterpret_cast<float4*>(&part[warp][(i * 32 + lane) * 8]);
        q[0] = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
        q[1] = make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.d; c += 32 * kWarpRows) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarpRows; ++w) s += part[w][c];
        p.partials[static_cast<int64_t>(blockIdx.x) * p.d + c] = s;
    }
}

// dgamma from the CTAs' partials: 32 columns per CTA, 32 threads per column each
// adding every 32nd partial in order, then the 32 in order.
__global__ void __launch_bounds__(1024) dgamma_kernel(const float* partials, int parts, int d, int accumulate,
                                                      float* dgamma) {
    __shared__ float red[32][33];
    wait_for_earlier_kernels();
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    float s = 0.f;
#pragma unroll 10
    for (int k = g; k < parts; k += 32) s += partials[static_cast<int64_t>(k) * d + col];
    red[g][c] = s;
    __syncthreads();
    if (g == 0) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += red[k][c];
        dgamma[col] = accumulate ? dgamma[col] + t : t;
    }
}

// ---------------------------------------------------------------------------
// Heads: norm and rotation in one pass.
//
// A pair's angle is positions[row] * freq[i].  In turns, as fixed point with 2^64
// for a whole one, the product in 64-bit integers drops whole turns by wrapping, so
// the fraction is off by the table's own error times the position and by the 2^-32 of a
// turn below the bits that are kept.  The table's error is 2^-65 of a turn by its fixed point and
// up to about 2^-55 by rope_turns' doubles for the fastest pair (less as the pairs slow down):
// 2^-35 of a turn at the millionth token, where a product in fp32 would be off by 0.06
// radians.  The quarter turn is split off as an integer too; sin and cos see at most an
// eighth of a turn.
//
// The pairs of a head lie in vectors of W elements: vector pair v is the W first and
// the W second elements of pairs (halves), or two vectors of adjacent pairs; past
// the rotated part, two vectors of the rest.  A thread holds 8 / W vector pairs, so a
// pair never leaves its thread and in-place work is safe; a head takes as many
// neighbouring lanes as that needs, a warp as many heads as fit (head_dim 96: 5 heads
// of 6 lanes).  W is the widest that divides the head, its rotated part, strides
// and addresses.  Arithmetic goes two pairs at a time: one by one, with a division
// per head and a 64-bit multiplication per address, the kernel issued 31 instructions
// per element where memory leaves time for 21 (8192 x 80 heads of 128 bf16: 100 us).
//
// Memory-bound.  8192 x 80 heads of 128 bf16: 55.8 us (6.0 TB/s, 0.89 of the measured copy
// rate; 32768 rows 0.98), gradient with both gammas' 83.5 us (0.89; 0.96); fp32 56.6 and
// 79.6 us at 4096 rows.  Heads whose vectors are 8 bytes are bound by the instructions of their many
// small pieces (72 elements: 47.2 and 73.2 us, floors 27.8 and 41.7); one token's 40 heads by
// latency (2.7 us).
// ---------------------------------------------------------------------------
constexpr int kHeadThreads = 256;
// A row's angles take a CTA as long as this many heads (16384 rows of 32 + 8 heads of 128 bf16,
// gradient: 92.6 us counting none, 88.6 one, 84.9 two, 87.3 five).
constexpr int kAngles = 2;
constexpr int kHeadSmem = 113 * 1024;  // at most: two CTAs per SM

// A thread's 8 first and 8 second elements of pairs.
struct HeadPairs {
    float2 a[4], b[4];
};

// Where a lane's vector pairs lie in a head.
template <int W, bool PAIRS>
struct HeadPlace {
    static constexpr int V = 8 / W;
    int a[V], b[V];   // first elements of the two vectors
    int v[V];         // place in the planes of the tables
    int all;          // vector pairs of a head
    int mine;         // this lane's vector pairs (with W = 8 always one, with 4 one or two)
    __device__ __forceinline__ HeadPlace(const HeadArgs& p, int lane) : all(p.dim / (2 * W)), mine((all - lane + p.lanes - 1) / p.lanes) {
        const int turned = p.rot / (2 * W);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = min(lane + k * p.lanes, all - 1);
            v[k] = i;
            if (i >= turned) {
                a[k] = p.rot + W * (i - turned);
                b[k] = a[k] + (p.dim - p.rot) / 2;
            } else if (W == 1 && PAIRS) {
                a[k] = 2 * i;
                b[k] = a[k] + 1;
            } else {
                a[k] = W * i;
                b[k] = a[k] + p.rot / 2;
            }
        }
    }
    __device__ __forceinline__ bool live(int k) const { return V == 1 || (V == 2 && k == 0) || k < mine; }
    // element of the head that is pair e's first (second: the one after it, or as far on in b)
    __device__ __forceinline__ int first(int k, int e) const {
        return !PAIRS || W == 1 ? a[k] + e : e < W / 2 ? a[k] + 2 * e : b[k] + 2 * e - W;
    }
    __device__ __forceinline__ int second(int k, int e) const { return !PAIRS || W == 1 ? b[k] + e : first(k, e) + 1; }
};

// A thread's part of a head as loaded.
template <bool F32, int W, bool PAIRS>
struct HeadRaw {
    static constexpr int V = 8 / W;
    RowVec<F32, W> a[V], b[V];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < V; ++k) a[k].clear(), b[k].clear();
    }
    __device__ __forceinline__ void load(const HeadPlace<W, PAIRS>& at, const char* head) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (at.live(k)) {
                a[k].load(head, at.a[k]);
                b[k].load(head, at.b[k]);
            }
    }
    __device__ __forceinline__ void get(HeadPairs& x) const {
        float first[8], second[8];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float u[W], v[W];
            a[k].get(u);
            b[k].get(v);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                first[k * W + e] = !PAIRS || W == 1 ? u[e] : e < W / 2 ? u[(2 * e) % W] : v[(2 * e) % W];
                second[k * W + e] = !PAIRS || W == 1 ? v[e] : e < W / 2 ? u[(2 * e + 1) % W] : v[(2 * e + 1) % W];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x.a[j] = make_float2(first[2 * j], first[2 * j + 1]);
            x.b[j] = make_float2(second[2 * j], second[2 * j + 1]);
        }
    }
    static __device__ __forceinline__ void put(const HeadPlace<W, PAIRS>& at, char* head, const HeadPairs& x) {
        float first[8], second[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            first[2 * j] = x.a[j].x, first[2 * j + 1] = x.a[j].y;
            second[2 * j] = x.b[j].x, second[2 * j + 1] = x.b[j].y;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (!at.live(k)) continue;
            float u[W], v[W];
#pragma unroll
            for (int e = 0; e < W; ++e) {
                if (!PAIRS || W == 1) {
                    u[e] = first[k * W + e];
                    v[e] = second[k * W + e];
                } else {
                    u[e] = e & 1 ? second[k * W + e / 2] : first[k * W + e / 2];
                    v[e] = e & 1 ? second[k * W + W / 2 + e / 2] : first[k * W + W / 2 + e / 2];
                }
            }
            RowVec<F32, W>::put(head, at.a[k], u);
            RowVec<F32, W>::put(head, at.b[k], v);
        }
    }
};

// A thread's parts of the heads it is going to work on, on their way into its own place
// in shared memory (asynchronous copies; a thread waits for its own): D of them under
// way and one that is read.  With one in registers instead, 32 KB under way on an SM, the
// gradient of 8192 x 80 heads of 128 bf16 took 109 us, not 84.  Vectors of 2 bytes, which such
// copies do not take, go through registers.
template <bool F32, int W, bool PAIRS, int D>
struct HeadRing {
    static constexpr int kVec = W * (F32 ? 4 : 2), kPiece = kVec < 16 ? kVec : 16, V = 8 / W, kPieces = kVec / kPiece;
    static constexpr bool kAsync = kVec >= 4;
    static constexpr int kStages = kAsync ? D + 1 : 0, kAhead = kAsync ? D : 1;
    static constexpr int kStageBytes = 2 * V * kVec * kHeadThreads;
    static constexpr int kBytes = kStages * kStageBytes;
    HeadRaw<F32, W, PAIRS> held;  // registers only
    uint32_t put_at, get_at, begin, end;

    __device__ __forceinline__ HeadRing(char* smem) {
        held.clear();
        begin = smem_u32(smem) + threadIdx.x * kPiece;
        end = begin + kBytes;
        put_at = get_at = begin;
    }
    static __device__ __forceinline__ void copy(uint32_t to, const char* from) {
        if constexpr (kPiece == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(kPiece < 4 ? 4 : kPiece) : "memory");
    }
    // the next head, if it is `there`
    __device__ __forceinline__ void put(const HeadPlace<W, PAIRS>& at, const char* head, bool there) {
        if constexpr (!kAsync) {
            if (there) held.load(at, head);
        } else {
            if (there) {
                constexpr int es = F32 ? 4 : 2;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (!at.live(k)) continue;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        copy(put_at + ((2 * k) * kPieces + i) * kPiece * kHeadThreads, head + at.a[k] * es + i * kPiece);
                        copy(put_at + ((2 * k + 1) * kPieces + i) * kPiece * kHeadThreads, head + at.b[k] * es + i * kPiece);
                    }
                }
            }
            put_at += kStageBytes;
            if (put_at == end) put_at = begin;
        }
    }
    __device__ __forceinline__ void get(const HeadPlace<W, PAIRS>& at, HeadRaw<F32, W, PAIRS>& x) {
        if constexpr (!kAsync) {
            x = held;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (!at.live(k)) {  // nothing was copied there
                    x.a[k].clear();
                    x.b[k].clear();
                    continue;
                }
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    piece(get_at + ((2 * k) * kPieces + i) * kPiece * kHeadThreads, x.a[k].w + i * (kPiece / 4));
                    piece(get_at + ((2 * k + 1) * kPieces + i) * kPiece * kHeadThreads, x.b[k].w + i * (kPiece / 4));
                }
            }
            get_at += kStageBytes;
            if (get_at == end) get_at = begin;
        }
    }
    static __device__ __forceinline__ void piece(uint32_t from, uint32_t* w) {
        if constexpr (kPiece == 16)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from) : "memory");
        else if constexpr (kPiece == 8)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(from) : "memory");
        else asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(from) : "memory");
    }
};
// One head of each ring is a group of copies; the oldest one's have arrived once no more
// than the ones ahead of it are under way.
__device__ __forceinline__ void head_copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void head_copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
template <bool F32>
constexpr int kHeadAhead = F32 ? 2 : 3;
template <bool F32>
constexpr int kHeadGradAhead = F32 ? 1 : 3;  // of each of its two rings

// Tables in shared memory hold two values for each pair of a head, dim floats: all
// first ones, then all second ones; each in planes of M pairs of every vector pair, so
// that neighbouring lanes read neighbouring M floats.
template <int W>
__device__ __forceinline__ int head_plane(int v, int e, int all) {
    constexpr int M = W < 4 ? W : 4;
    return ((e / M) * all + v) * M + e % M;
}
template <int W, bool PAIRS>
__device__ __forceinline__ void head_planes(const HeadPlace<W, PAIRS>& at, const float* table, int dim, HeadPairs& x) {
    constexpr int M = W < 4 ? W : 4, V = 8 / W;
    float c[8], s[8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int h = 0; h < W / M; ++h) {
            const float* from = table + (h * at.all + at.v[k]) * M;
            float* ck = c + k * W + h * M;
            float* sk = s + k * W + h * M;
            if constexpr (M == 4) {
                const float4 u = *reinterpret_cast<const float4*>(from), v = *reinterpret_cast<const float4*>(from + dim / 2);
                ck[0] = u.x, ck[1] = u.y, ck[2] = u.z, ck[3] = u.w;
                sk[0] = v.x, sk[1] = v.y, sk[2] = v.z, sk[3] = v.w;
            } else if constexpr (M == 2) {
                const float2 u = *reinterpret_cast<const float2*>(from), v = *reinterpret_cast<const float2*>(from + dim / 2);
                ck[0] = u.x, ck[1] = u.y;
                sk[0] = v.x, sk[1] = v.y;
            } else {
                ck[0] = *from;
                sk[0] = from[dim / 2];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x.a[j] = make_float2(c[2 * j], c[2 * j + 1]);
        x.b[j] = make_float2(s[2 * j], s[2 * j + 1]);
    }
}

// sin and cos of pi y, |y| <= 1/4: their Taylor series to y^9 and y^10, off by less than
// (pi / 4)^11 / 11! = 2^-29 and (pi / 4)^12 / 12! = 2^-33 there; pi in two parts, so that the sine keeps
// its last bit.
__device__ __forceinline__ void sincos_eighth(float y, float& s, float& c) {
    const float z = y * y;
    float u = fmaf(z, 0.08214588661f, -0.59926452932f);
    u = fmaf(u, z, 2.55016403988f);
    u = fmaf(u, z, -5.16771278005f);
    s = fmaf(y, 3.14159274101f, y * fmaf(u, z, -8.74227801e-8f));
    float v = fmaf(z, -0.02580689139f, 0.23533063036f);
    v = fmaf(v, z, -1.33526276885f);
    v = fmaf(v, z, 4.05871212642f);
    v = fmaf(v, z, -4.93480220054f);
    c = fmaf(v, z, 1.f);
}

// cos and sin of `tokens` positions, every apart-th, scaled (1 and 0 past the rotated part, read
// there but not used): a table of dim floats for each, the first one's at `place` of `places` in a
// circle.
template <int W, bool PAIRS>
__device__ __forceinline__ void head_angles(const HeadArgs& p, const int64_t* positions, int64_t apart, int tokens, float* tables, int place, int places) {
    const int half = p.dim / 2, pairs = p.rot / 2, turned = p.rot / (2 * W), all = p.dim / (2 * W);
    int t = threadIdx.x / half, c = threadIdx.x - t * half;  // pair c of row t
    const int t_on = kHeadThreads / half, c_on = kHeadThreads - t_on * half;
    while (t < tokens) {
        float cs = 1.f, sn = 0.f;
        int v = c / W, e = c - v * W;
        if (c < pairs) {
            if (W > 1 && PAIRS) {  // a vector holds W / 2 pairs; the second vector's follow the first's
                constexpr int P = W > 1 ? W / 2 : 1;
                const int vec = c / P, in = c - vec * P;
                v = vec < turned ? vec : vec - turned;
                e = vec < turned ? in : P + in;
            }
            const uint64_t turn = static_cast<uint64_t>(positions[t * apart]) * p.turns[c];
            const uint32_t hi = static_cast<uint32_t>(turn >> 32);
            const uint32_t quarter = (hi + 0x20000000u) >> 30;
            const int32_t rest = static_cast<int32_t>(hi - (quarter << 30));  // an eighth of a turn at most
            float s, k;
            sincos_eighth(static_cast<float>(rest) * 0x1p-31f, s, k);
            const float cq = quarter & 1 ? s : k, sq = quarter & 1 ? k : s;
            cs = ((quarter + 1) & 2 ? -cq : cq) * p.scale;
            sn = (quarter & 2 ? -sq : sq) * p.scale;
        }
        const int at = place + t;
        float* to = tables + (at < places ? at : at - places) * p.dim + head_plane<W>(v, e, all);
        to[0] = cs;
        to[half] = sn;
        t += t_on;
        c += c_on;
        if (c >= half) c -= half, ++t;
    }
}

// Turns the pairs by the row's angles, or back.  A vector pair is turned as a whole or not at
// all; one past the rotated part keeps its bits: a product with cos = 1 and sin = 0 made
// the partner of an infinity NaN.  (Chosen after the arithmetic: branches around it spilled at 4
// elements per vector, 72 elements 51.5 us against 46.9 without any choice.)
template <int W, bool PAIRS, bool BACK>
__device__ __forceinline__ void head_turn(const HeadArgs& p, const HeadPlace<W, PAIRS>& at, const float* row, HeadPairs& x) {
    const int turned = p.rot / (2 * W);
    if (W == 8 && at.v[0] >= turned) return;
    HeadPairs w;
    head_planes(at, row, p.dim, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool on0 = at.v[2 * j / W] < turned, on1 = at.v[(2 * j + 1) / W] < turned;
        const float2 ac = mul2(x.a[j], w.a[j]), bc = mul2(x.b[j], w.a[j]);
        float2 a, b;
        // the side that subtracts in single instructions, which negate for free
        if (BACK) {
            a = fma2(x.b[j], w.b[j], ac);
            b = make_float2(fmaf(-x.a[j].x, w.b[j].x, bc.x), fmaf(-x.a[j].y, w.b[j].y, bc.y));
        } else {
            b = fma2(x.a[j], w.b[j], bc);
            a = make_float2(fmaf(-x.b[j].x, w.b[j].x, ac.x), fmaf(-x.b[j].y, w.b[j].y, ac.y));
        }
        x.a[j] = make_float2(on0 ? a.x : x.a[j].x, on1 ? a.y : x.a[j].y);
        x.b[j] = make_float2(on0 ? b.x : x.b[j].x, on1 ? b.y : x.b[j].y);
    }
}

// gamma as a table, copied by the CTA's first head's lanes (asynchronously: in the group
// of the first head's copies).  (In registers it cost 16
// of them, and a CTA per SM.)
template <int W, bool PAIRS>
__device__ __forceinline__ void head_gamma(const HeadPlace<W, PAIRS>& at, const float* gamma, int dim, float* table) {
#pragma unroll
    for (int k = 0; k < 8 / W; ++k)
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const uint32_t to = smem_u32(table + head_plane<W>(at.v[k], e, at.all));
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(gamma + at.first(k, e)) : "memory");
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + dim * 2), "l"(gamma + at.second(k, e)) : "memory");
        }
}

// Sum over a head's lanes, the same in each: a head's lanes are neighbours, `lane` this
// one's place among them; whole warps come here.
__device__ __forceinline__ float head_sum(float v, int lane, int lanes) {
    if (lanes == 8) {
#pragma unroll
        for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    if ((lanes & (lanes - 1)) == 0) {
        for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        if (o >= lanes) continue;
        const float t = __shfl_down_sync(0xffffffffu, v, o);
        // a tree over any number: the upper part of what is left is folded onto its beginning
        if (lane + o < lanes && lane < o) v += t;
    }
    return __shfl_sync(0xffffffffu, v, (threadIdx.x & 31) - lane);
}

// 1 / sqrt(sum / dim + eps): the hardware's approximation and a Newton step.
__device__ __forceinline__ float head_rstd(float sum, float inv_dim, float eps) {
    const float a = fmaf(sum, inv_dim, eps), y = rsqrtf(a);
    const float e = fmaf(-a * y, y, 1.f);
    return a > 1e-35f && a < 1e35f ? fmaf(0.5f * y, e, y) : y;
}

// This thread's way through its CTA's rows: every ranges-th of them, so that all CTAs
// read and write in the same part of memory; of their (row, head) items it takes every
// stride-th.  All strides are the host's.
struct HeadWay {
    int lane;          // of its head
    int slot;          // which head of the CTA's round; -1: a lane that is left over
    int row, head;     // its first item, among the CTA's rows
    int rows;          // of the CTA
    int64_t tok0;
    int64_t rounds;    // that all threads of the CTA make
    __device__ __forceinline__ HeadWay(const HeadArgs& p, const HeadGroup& g) {
        const int local = static_cast<int>(blockIdx.x) - g.cta0, range = local / g.split, part = local - range * g.split;
        const int per_warp = 32 / p.lanes, in_warp = (threadIdx.x & 31) / p.lanes;
        lane = (threadIdx.x & 31) - in_warp * p.lanes;
        slot = in_warp < per_warp ? (threadIdx.x >> 5) * per_warp + in_warp : -1;
        const int item = part * g.slots + max(slot, 0);
        row = item / g.heads;
        head = item - row * g.heads;
        tok0 = range;
        rows = static_cast<int>((p.rows - range + g.ranges - 1) / g.ranges);
        rounds = max(static_cast<int64_t>(0), (static_cast<int64_t>(rows) * g.heads - part * g.slots + g.stride - 1) / g.stride);
    }
};
// The CTA's positions, in shared memory where they are few enough (copied with the
// first head; else nullptr): read from memory at every step, they held up a CTA of 8 heads, whose
// steps are short (16384 rows of 32 + 8 heads bf16: gradient 114 us).
constexpr int kHeadPositions = 1024;
__device__ __forceinline__ const int64_t* head_positions(const HeadArgs& p, const HeadGroup& g, const HeadWay& way, float* smem) {
    const int64_t* from = p.positions + way.tok0;
    if (!p.rot || !g.held) return nullptr;
    for (int i = threadIdx.x; i < way.rows; i += kHeadThreads)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(smem) + 8 * i), "l"(from + static_cast<int64_t>(i) * g.ranges) : "memory");
    return reinterpret_cast<const int64_t*>(smem);
}

// Rows that the rounds up to a step's end reach: the angles of those of the next step are
// made while this one's are read, in a circle of g.places tables.
struct HeadReach {
    int rows, rest, place;  // whole rows and heads of one more; where the next row's table goes
    __device__ __forceinline__ HeadReach() : rows(0), rest(0), place(0) {}
    template <int W, bool PAIRS>
    __device__ __forceinline__ void step(const HeadArgs& p, const HeadGroup& g, const HeadWay& way, const int64_t* positions, float* tables) {
        const int before = min(way.rows, rows + (rest > 0));
        rows += g.step_rows;
        rest += g.step_heads;
        if (rest >= g.heads) rest -= g.heads, ++rows;
        rows = min(rows, way.rows);  // (stays there: no overflow)
        const int more = min(way.rows, rows + (rest > 0)) - before;
        if (positions) head_angles<W, PAIRS>(p, positions + before, 1, more, tables, place, g.places);
        else head_angles<W, PAIRS>(p, p.positions + way.tok0 + static_cast<int64_t>(before) * g.ranges, g.ranges, more, tables, place, g.places);
        place += more;
        if (place >= g.places) place -= g.places;
    }
};

// Forward, persistent.  The group is known when it is compiled: its strides are then
// constants of the launch, where an index into the groups loaded 16 words for each head
// and round.
template <bool F32, int W, bool PAIRS, int G>
__device__ __forceinline__ void head_body(const HeadArgs& p) {
    using Ring = HeadRing<F32, W, PAIRS, kHeadAhead<F32>>;
    extern __shared__ __align__(16) float smem[];  // the ring, gamma, angles
    constexpr int64_t es = F32 ? 4 : 2;
    const HeadGroup& g = p.g[G];
    const HeadWay way(p, g);
    const HeadPlace<W, PAIRS> at(p, way.lane);
    const int rows = way.slot < 0 ? 0 : way.rows;
    int row = way.row, head = way.head, row1 = way.row, head1 = way.head;  // 1: of the copies
    const char* in = static_cast<const char*>(g.in) + ((way.tok0 + static_cast<int64_t>(row) * g.ranges) * g.in_row + head * g.in_head) * es;
    char* out = static_cast<char*>(g.out) + ((way.tok0 + static_cast<int64_t>(row) * g.ranges) * g.out_row + head * g.out_head) * es;
    Ring ring(reinterpret_cast<char*>(smem));
    const auto ahead = [&] {
        ring.put(at, in, row1 < rows);
        head_copies_commit();
        row1 += g.rows_on;
        head1 += g.heads_on;
        in += g.in_step;
        if (head1 >= g.heads) head1 -= g.heads, ++row1, in += g.in_wrap;
    };
    float* gammas = smem + Ring::kBytes / 4;
    float* tables = gammas + (p.dim + 3) / 4 * 4;
    float* after = tables + (g.places * p.dim + 3) / 4 * 4;
    const int64_t* positions = head_positions(p, g, way, after);
    const float inv_dim = 1.f / static_cast<float>(p.dim);
    const bool norm = g.gamma != nullptr;
    if (norm && way.slot == 0) head_gamma(at, g.gamma, p.dim, gammas);
#pragma unroll
    for (int d = 0; d < Ring::kAhead; ++d) ahead();
    head_copies_wait<Ring::kAhead - 1>();  // gamma and the positions
    __syncthreads();
    HeadReach reach;
    if (p.rot) reach.step<W, PAIRS>(p, g, way, positions, tables);
    int place = row;  // of its row's angles (a first item's row is among the first step's)
    // whole warps stay in the loops: a head's sum is over lanes
    for (int64_t left = way.rounds; left > 0; left -= g.rounds) {
        __syncthreads();  // this step's angles are there, the one's before have been read
        if (p.rot && left > g.rounds) reach.step<W, PAIRS>(p, g, way, positions, tables);
        for (int r = static_cast<int>(min(static_cast<int64_t>(g.rounds), left)); r > 0; --r) {
            HeadRaw<F32, W, PAIRS> raw;
            HeadPairs x;
            if constexpr (Ring::kAsync) {
                head_copies_wait<Ring::kAhead - 1>();
                ahead();
                ring.get(at, raw);
            } else {
                ring.get(at, raw);
                ahead();
            }
            raw.get(x);
            const bool live = row < rows;
            if (norm) {
                float2 sq = mul2(x.a[0], x.a[0]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j) sq = fma2(x.a[j], x.a[j], sq);
                    sq = fma2(x.b[j], x.b[j], sq);
                }
                const float2 rstd = both2(head_rstd(head_sum(sq.x + sq.y, way.lane, p.lanes), inv_dim, p.eps));
                HeadPairs gamma;
                head_planes(at, gammas, p.dim, gamma);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x.a[j] = mul2(mul2(x.a[j], rstd), gamma.a[j]);
                    x.b[j] = mul2(mul2(x.b[j], rstd), gamma.b[j]);
                }
            }
            if (live) {
                if (p.rot) head_turn<W, PAIRS, false>(p, at, tables + place * p.dim, x);
                HeadRaw<F32, W, PAIRS>::put(at, out, x);
            }
            row += g.rows_on;
            place += g.rows_on;
            head += g.heads_on;
            out += g.out_step;
            if (head >= g.heads) head -= g.heads, ++row, ++place, out += g.out_wrap;
            if (place >= g.places) place -= g.places;
        }
    }
}

template <bool F32, int W, bool PAIRS>
__global__ void __launch_bounds__(kHeadThreads, W < 4 ? 2 : F32 ? 3 : 4) head_kernel(const __grid_constant__ HeadArgs p) {
    wait_for_earlier_kernels();
    if (static_cast<int>(blockIdx.x) < p.g[1].cta0) head_body<F32, W, PAIRS, 0>(p);
    else head_body<F32, W, PAIRS, 1>(p);
}

// Gradient.  With t = dy turned back, u = t gamma, S1 = sum x^2 and S2 = sum u x, both
// in the same round of shuffles: dx = r u - x r^3 S2 / dim.  A thread keeps its
// elements' part of dgamma in registers; the slots' parts are added at the end in order.
template <bool F32, int W, bool PAIRS, int G>
__device__ __forceinline__ void head_grad_body(const HeadArgs& p) {
    using Ring = HeadRing<F32, W, PAIRS, kHeadGradAhead<F32>>;
    extern __shared__ __align__(16) float smem[];  // the rings of dy and x, gamma, angles
    constexpr int64_t es = F32 ? 4 : 2;
    const HeadGroup& g = p.g[G];
    const HeadWay way(p, g);
    const HeadPlace<W, PAIRS> at(p, way.lane);
    const bool norm = g.gamma != nullptr;
    const int rows = way.slot < 0 ? 0 : way.rows;
    int row = way.row, head = way.head, row1 = way.row, head1 = way.head;  // 1: of the copies
    const char* in = static_cast<const char*>(g.in) + ((way.tok0 + static_cast<int64_t>(row) * g.ranges) * g.in_row + head * g.in_head) * es;
    const char* from = static_cast<const char*>(g.x) + ((way.tok0 + static_cast<int64_t>(row) * g.ranges) * g.x_row + head * g.x_head) * es;
    char* out = static_cast<char*>(g.out) + ((way.tok0 + static_cast<int64_t>(row) * g.ranges) * g.out_row + head * g.out_head) * es;
    Ring dys(reinterpret_cast<char*>(smem)), xs(reinterpret_cast<char*>(smem) + Ring::kBytes);
    const auto ahead = [&] {
        dys.put(at, in, row1 < rows);
        xs.put(at, from, norm && row1 < rows);
        head_copies_commit();
        row1 += g.rows_on;
        head1 += g.heads_on;
        in += g.in_step;
        from += g.x_step;
        if (head1 >= g.heads) head1 -= g.heads, ++row1, in += g.in_wrap, from += g.x_wrap;
    };
    float* gammas = smem + 2 * Ring::kBytes / 4;
    float* tables = gammas + (p.dim + 3) / 4 * 4;
    float* after = tables + (g.places * p.dim + 3) / 4 * 4;
    const int64_t* positions = head_positions(p, g, way, after);
    const float inv_dim = 1.f / static_cast<float>(p.dim);
    if (norm && way.slot == 0) head_gamma(at, g.gamma, p.dim, gammas);
#pragma unroll
    for (int d = 0; d < Ring::kAhead; ++d) ahead();
    head_copies_wait<Ring::kAhead - 1>();  // gamma and the positions
    __syncthreads();
    HeadReach reach;
    if (p.rot) reach.step<W, PAIRS>(p, g, way, positions, tables);
    int place = row;
    HeadPairs dg;
#pragma unroll
    for (int j = 0; j < 4; ++j) dg.a[j] = dg.b[j] = both2(0.f);
    for (int64_t left = way.rounds; left > 0; left -= g.rounds) {
        __syncthreads();  // this step's angles are there, the one's before have been read
        if (p.rot && left > g.rounds) reach.step<W, PAIRS>(p, g, way, positions, tables);
        for (int n = static_cast<int>(min(static_cast<int64_t>(g.rounds), left)); n > 0; --n) {
            HeadPairs t, h;
            {
                HeadRaw<F32, W, PAIRS> dy, x;
                if constexpr (Ring::kAsync) {
                    head_copies_wait<Ring::kAhead - 1>();
                    ahead();
                    dys.get(at, dy);
                    xs.get(at, x);
                } else {
                    dys.get(at, dy);
                    xs.get(at, x);
                    ahead();
                }
                dy.get(t);
                x.get(h);
            }
            const bool live = row < rows;
            if (p.rot && live) head_turn<W, PAIRS, true>(p, at, tables + place * p.dim, t);
            if (norm) {
                float2 s1 = both2(0.f), s2 = both2(0.f);
                HeadPairs u;
                head_planes(at, gammas, p.dim, u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u.a[j] = mul2(t.a[j], u.a[j]);
                    u.b[j] = mul2(t.b[j], u.b[j]);
                    s1 = fma2(h.a[j], h.a[j], fma2(h.b[j], h.b[j], s1));
                    s2 = fma2(u.a[j], h.a[j], fma2(u.b[j], h.b[j], s2));
                }
                const float sq = head_sum(s1.x + s1.y, way.lane, p.lanes), dot = head_sum(s2.x + s2.y, way.lane, p.lanes);
                const float r = head_rstd(sq, inv_dim, p.eps);
                const float2 back = both2(-r * (r * dot * inv_dim)), r2 = both2(r);
                if (live) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        h.a[j] = mul2(h.a[j], r2);
                        h.b[j] = mul2(h.b[j], r2);
                        dg.a[j] = fma2(t.a[j], h.a[j], dg.a[j]);
                        dg.b[j] = fma2(t.b[j], h.b[j], dg.b[j]);
                        t.a[j] = fma2(h.a[j], back, mul2(u.a[j], r2));
                        t.b[j] = fma2(h.b[j], back, mul2(u.b[j], r2));
                    }
                }
            }
            if (live) HeadRaw<F32, W, PAIRS>::put(at, out, t);
            row += g.rows_on;
            place += g.rows_on;
            head += g.heads_on;
            out += g.out_step;
            if (head >= g.heads) head -= g.heads, ++row, ++place, out += g.out_wrap;
            if (place >= g.places) place -= g.places;
        }
    }
    if (!g.partials) return;
    // [slots][dim] over all of it, then the slots in order
    head_copies_wait<0>();
    __syncthreads();
    if (way.slot >= 0) {
#pragma unroll
        for (int k = 0; k < 8 / W; ++k)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const int j = (k * W + e) / 2;
                if (!at.live(k)) continue;
                smem[way.slot * p.dim + at.first(k, e)] = (k * W + e) & 1 ? dg.a[j].y : dg.a[j].x;
                smem[way.slot * p.dim + at.second(k, e)] = (k * W + e) & 1 ? dg.b[j].y : dg.b[j].x;
            }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.dim; c += kHeadThreads) {
        float s = 0.f;
#pragma unroll 8
        for (int w = 0; w < g.slots; ++w) s += smem[w * p.dim + c];
        g.partials[static_cast<int64_t>(static_cast<int>(blockIdx.x) - g.cta0) * p.dim + c] = s;
    }
}

template <bool F32, int W, bool PAIRS>
__global__ void __launch_bounds__(kHeadThreads, W == 1 ? 1 : 2) head_grad_kernel(const __grid_constant__ HeadArgs p) {
    wait_for_earlier_kernels();
    if (static_cast<int>(blockIdx.x) < p.g[1].cta0) head_grad_body<F32, W, PAIRS, 0>(p);
    else head_grad_body<F32, W, PAIRS, 1>(p);
}

// dgamma of every group from its CTAs' partials, as dgamma_kernel does.
__global__ void __launch_bounds__(1024) head_dgamma_kernel(const __grid_constant__ HeadArgs p) {
    __shared__ float red[32][33];
    wait_for_earlier_kernels();
    const HeadGroup& g = p.g[blockIdx.y];
    if (!g.dgamma) return;
    const int c = threadIdx.x & 31, k0 = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    float s = 0.f;
    if (col < p.dim && g.partials)
#pragma unroll 10
        for (int k = k0; k < g.ranges; k += 32) s += g.partials[static_cast<int64_t>(k) * p.dim + col];
    red[k0][c] = s;
    __syncthreads();
    if (k0 == 0 && col < p.dim) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += red[k][c];
        g.dgamma[col] = g.accumulate ? g.dgamma[col] + t : t;
    }
}

template <bool F32>
cudaError_t launch_fwd(const RmsArgs& a, cudaStream_t st) {
    const unsigned rows = static_cast<unsigned>((a.rows + 127) / 128 * 128);
    note_launch();
    if (a.d <= kWarpMaxD) {
        const unsigned grid = rows / kWarpRows;
        if (a.d <= 256) return launch_early(rmsnorm_kernel<F32, 1, true>, grid, 32 * kWarpRows, 0, st, a);
        else if (a.d <= 512) return launch_early(rmsnorm_kernel<F32, 2, true>, grid, 32 * kWarpRows, 0, st, a);
        else return launch_early(rmsnorm_kernel<F32, 4, true>, grid, 32 * kWarpRows, 0, st, a);
    } else {
        // two vectors per thread up to 8192 columns (8192 x 4096 bf16: 40.9 us with one, 30.8 with two)
        const int v = a.d <= 8192 ? 2 : 4;
        const int threads = ((a.d / 8 + v - 1) / v + 31) / 32 * 32;
        if (v == 2) return launch_early(rmsnorm_kernel<F32, 2, false>, rows, threads, 0, st, a);
        else return launch_early(rmsnorm_kernel<F32, 4, false>, rows, threads, 0, st, a);
    }
}

template <bool F32, int V, int T, int B>
cudaError_t launch_grad(RmsGradArgs a, int parts, int stage, cudaStream_t st) {
    constexpr int ring = kGradRing / B;
    a.stages = std::min(kMaxGradStages, ring / stage);
    static PerDevice done;
    const cudaError_t e = allow_smem(rmsnorm_grad_kernel<F32, V, T, B>, ring, done);
    if (e != cudaSuccess) return e;
    const int threads = ((a.d / 8 + V - 1) / V + 31) / 32 * 32;
    note_launch();
    return launch_early(rmsnorm_grad_kernel<F32, V, T, B>, parts, threads, a.stages * stage, st, a);
}

template <bool F32>
cudaError_t launch_bwd(const RmsGradArgs& a0, cudaStream_t st) {
    RmsGradArgs a = a0;
    a.err = device_error_word();
    a.inject = inject_mx_timeout();
    // Two CTAs per SM where half the ring still holds two rows: one computes while
    // the other stands at its barrier (8192 x 5120 bf16: 71 us with one, 55 with two).
    const int stage = a.d * (F32 ? 4 : 2) * (a.dres ? 3 : 2);
    // Up to 8192 columns that is always so in bf16, up to 4096 in fp32.
    static_assert(2 * 8192 * 2 * 3 <= kGradRing / 2 && 2 * 4096 * 4 * 3 <= kGradRing / 2, "two rows in half the ring");
    const bool two = a.d <= 8192 && 2 * stage <= kGradRing / 2;
    const int most = rmsnorm_grad_parts(a.rows, a.d);
    const int parts = a.d <= kWarpMaxD ? most : std::min(most, (two ? 2 : 1) * device_sm_count());
    if (parts) {
        cudaError_t e = cudaSuccess;
        // Up to 5120 columns 320 threads hold two vectors each; told so, the compiler has
        // the registers to keep gamma (8192 x 5120 bf16 55.0 us against 65.2 with the bound
        // of 512 threads, 4608 50.4 and 61.2, fp32 5120 without residual 92.3 and 136.7).
        if (a.d <= kWarpMaxD) {
            note_launch();
            const auto kernel = a.d <= 256   ? rmsnorm_grad_warp_kernel<F32, 1>
                                : a.d <= 512 ? rmsnorm_grad_warp_kernel<F32, 2>
                                             : rmsnorm_grad_warp_kernel<F32, 4>;
            e = launch_early(kernel, parts, 32 * kWarpRows, 0, st, a);
        } else if (a.d <= 4096) e = launch_grad<F32, 1, 512, 2>(a, parts, stage, st);
        else if (a.d > 8192) e = launch_grad<F32, 2, 1024, 1>(a, parts, stage, st);
        else if (F32 && !two) e = launch_grad<true, 2, 512, 1>(a, parts, stage, st);
        else if (a.d <= 5120) e = launch_grad<F32, 2, 320, 2>(a, parts, stage, st);
        else e = launch_grad<F32, 2, 512, 2>(a, parts, stage, st);
        if (e != cudaSuccess) return e;
    }
    note_launch();
    return launch_early(dgamma_kernel, a.d / 32, 1024, 0, st, a.partials, parts, a.d, a.accumulate, a.dgamma);
}

// A group's share of a launch's CTAs: by heads and the angles of its rows.
int64_t head_share(int64_t ctas, int heads, int all_heads, int groups) {
    return std::max<int64_t>(1, ctas * (heads + kAngles) / (all_heads + kAngles * groups));
}

// Lanes per head, 16 elements each, and heads in a CTA's round.
int head_lanes(int dim) { return (dim + 15) / 16; }
int head_slots(int lanes) { return kHeadThreads / 32 * (32 / lanes); }

// A group's CTAs and strides: `ctas` of them, fewer where there are fewer rows; with a
// CTA per row and more CTAs than that (split), a row's heads over several.  A step is
// kHeadRounds rounds, fewer where the angles of two steps' rows would take more than
// kHeadTables.  Returns the bytes of gamma, the angles and the positions.
constexpr int kHeadRounds = 4;
constexpr int kHeadTables = 18 * 1024;
int plan_group(HeadArgs& a, HeadGroup& g, int64_t ctas, int64_t es, bool split, int64_t* used) {
    g.slots = head_slots(a.lanes);
    g.ranges = static_cast<int32_t>(std::min<int64_t>(a.rows, ctas));
    const int rounds = (g.heads + g.slots - 1) / g.slots;  // of one row
    g.split = split ? static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(rounds, ctas / g.ranges))) : 1;
    g.stride = g.slots * g.split;
    g.rows_on = g.stride / g.heads;
    g.heads_on = g.stride - g.rows_on * g.heads;
    g.rounds = kHeadRounds;
    const auto places = [&] { return 2 * ((g.rounds * g.stride + g.heads - 1) / g.heads + 1); };
    while (g.rounds > 1 && a.rot && places() * a.dim * 4 > kHeadTables) g.rounds /= 2;
    g.places = places();
    g.step_rows = g.rounds * g.stride / g.heads;
    g.step_heads = g.rounds * g.stride - g.step_rows * g.heads;
    const auto steps = [&](int64_t row, int64_t head, int64_t* step, int64_t* wrap) {
        *step = (g.rows_on * g.ranges * row + g.heads_on * head) * es;
        *wrap = (g.ranges * row - g.heads * head) * es;
    };
    steps(g.in_row, g.in_head, &g.in_step, &g.in_wrap);
    steps(g.x_row, g.x_head, &g.x_step, &g.x_wrap);
    steps(g.out_row, g.out_head, &g.out_step, &g.out_wrap);
    g.cta0 = static_cast<int32_t>(*used);
    *used += static_cast<int64_t>(g.ranges) * g.split;
    const int64_t rows = (a.rows + g.ranges - 1) / g.ranges;  // of a CTA, at most
    g.held = rows <= kHeadPositions;
    return 4 * ((a.dim + 3) / 4 * 4 + (a.rot ? (g.places * a.dim + 3) / 4 * 4 : 0)) + (a.rot && g.held ? static_cast<int>(rows) * 8 : 0);
}

template <bool F32, int W, bool PAIRS>
cudaError_t run_heads(HeadArgs& a, cudaStream_t st) {
    a.lanes = head_lanes(a.dim);
    int64_t ctas = 0;
    int smem = 0;
    // As many CTAs as are resident, or several times as many where each still makes 16 rounds (of fp32 8):
    // memory serves waves of them faster than one of longer ones (32768 x 80 heads of 128 bf16: 240
    // us with one, 220 with two, 202 with six; 8192 of 64 29.7, 31.4 and 41.7).
    const int64_t resident = static_cast<int64_t>(W < 4 ? 2 : F32 ? 3 : 4) * device_sm_count();
    const int64_t most = resident * std::max<int64_t>(1, a.rows * a.all_heads / head_slots(a.lanes) / (F32 ? 8 : 16) / resident);
    for (int i = 0; i < a.n; ++i)
        smem = std::max(smem, plan_group(a, a.g[i], head_share(most, a.g[i].heads, a.all_heads, a.all_groups), F32 ? 4 : 2, true, &ctas));
    if (a.n == 1) a.g[1].cta0 = INT32_MAX;
    smem += HeadRing<F32, W, PAIRS, kHeadAhead<F32>>::kBytes;
    static PerDevice done;
    const cudaError_t e = allow_smem(head_kernel<F32, W, PAIRS>, kHeadSmem, done);
    if (e != cudaSuccess) return e;
    note_launch();
    return launch_early(head_kernel<F32, W, PAIRS>, static_cast<unsigned>(ctas), kHeadThreads, smem, st, a);
}

template <bool F32, int W, bool PAIRS>
cudaError_t run_heads_grad(HeadArgs& a, cudaStream_t st) {
    a.lanes = head_lanes(a.dim);
    int64_t ctas = 0;
    int wanted = 0, smem = 0;
    for (int i = 0; i < a.n; ++i) {
        HeadGroup& g = a.g[i];
        g.cta0 = static_cast<int32_t>(ctas);
        wanted += g.dgamma != nullptr;
        if (!g.heads || !a.rows) continue;  // an empty sum: no ranges
        smem = std::max(smem, plan_group(a, g, head_grad_parts(a.rows, g.heads, a.all_heads, a.all_groups), F32 ? 4 : 2, false, &ctas));
    }
    if (a.n == 1) a.g[1].cta0 = INT32_MAX;
    smem = std::max(smem + 2 * HeadRing<F32, W, PAIRS, kHeadGradAhead<F32>>::kBytes, head_slots(a.lanes) * a.dim * 4);
    if (ctas) {
        static PerDevice done;
        cudaError_t e = allow_smem(head_grad_kernel<F32, W, PAIRS>, kHeadSmem, done);
        if (e != cudaSuccess) return e;
        note_launch();
        e = launch_early(head_grad_kernel<F32, W, PAIRS>, static_cast<unsigned>(ctas), kHeadThreads, smem, st, a);
        if (e != cudaSuccess || !wanted) return e;
    }
    if (!wanted) return cudaSuccess;
    note_launch();
    return launch_early(head_dgamma_kernel, dim3((a.dim + 31) / 32, a.n), 1024, 0, st, a);
}

template <int N>
using Int = std::integral_constant<int, N>;

}  // namespace

int head_width(const HeadArgs& a, int64_t es) {
    for (int w = static_cast<int>(16 / es); w > 1; w /= 2) {
        bool ok = a.dim % (2 * w) == 0 && a.rot % (2 * w) == 0;
        const int64_t bytes = w * es;
        const auto fits = [&](const void* p, int64_t row, int64_t head) {
            return reinterpret_cast<uintptr_t>(p) % bytes == 0 && row * es % bytes == 0 && head * es % bytes == 0;
        };
        for (int i = 0; i < a.n; ++i)
            ok = ok && fits(a.g[i].in, a.g[i].in_row, a.g[i].in_head) && fits(a.g[i].x, a.g[i].x_row, a.g[i].x_head) &&
                 fits(a.g[i].out, a.g[i].out_row, a.g[i].out_head);
        if (ok) return w;
    }
    return 1;
}

int head_grad_parts(int64_t rows, int heads, int all_heads, int groups) {
    // all resident: 8192 x 80 heads of 128 bf16 84 us, with twice as many 90
    return static_cast<int>(std::min(rows, head_share(2 * static_cast<int64_t>(device_sm_count()), heads, all_heads, groups)));
}

namespace {

// run(width, f32, pairs) as types
template <class Run>
cudaError_t with_head_kind(const HeadArgs& a, int f32, const Run& run) {
    const auto layout = [&](auto width, auto is_f32) { return a.pairs ? run(width, is_f32, Int<1>{}) : run(width, is_f32, Int<0>{}); };
    if (f32) return a.width == 4 ? layout(Int<4>{}, Int<1>{}) : a.width == 2 ? layout(Int<2>{}, Int<1>{}) : layout(Int<1>{}, Int<1>{});
    return a.width == 8   ? layout(Int<8>{}, Int<0>{})
           : a.width == 4 ? layout(Int<4>{}, Int<0>{})
           : a.width == 2 ? layout(Int<2>{}, Int<0>{})
                          : layout(Int<1>{}, Int<0>{});
}

}  // namespace

cudaError_t launch_heads(HeadArgs a, int f32, cudaStream_t st) {
    return with_head_kind(a, f32, [&](auto w, auto f, auto pairs) {
        return run_heads<decltype(f)::value != 0, decltype(w)::value, decltype(pairs)::value != 0>(a, st);
    });
}

cudaError_t launch_heads_grad(HeadArgs a, int f32, cudaStream_t st) {
    return with_head_kind(a, f32, [&](auto w, auto f, auto pairs) {
        return run_heads_grad<decltype(f)::value != 0, decltype(w)::value, decltype(pairs)::value != 0>(a, st);
    });
}

int rmsnorm_grad_parts(int64_t rows, int64_t d) {
    const int64_t sms = device_sm_count();
    if (d <= kWarpMaxD) return static_cast<int>(std::min((rows + kWarpRows - 1) / kWarpRows, (d <= 256 ? 4 : 2) * sms));
    return static_cast<int>(std::min(rows, 2 * sms));
}

cudaError_t launch_rmsnorm(const RmsArgs& a, int f32, cudaStream_t st) {
    return f32 ? launch_fwd<true>(a, st) : launch_fwd<false>(a, st);
}

cudaError_t launch_rmsnorm_grad(const RmsGradArgs& a, int f32, cudaStream_t st) {
    return f32 ? launch_bwd<true>(a, st) : launch_bwd<false>(a, st);
}

}  // namespace hm
