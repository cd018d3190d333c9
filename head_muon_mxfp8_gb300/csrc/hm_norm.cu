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
// Far from it are the gradient's fp32 forms whose registers spill: 8192 rows of 6656
// columns without a residual's gradient 183 us (3.6 TB/s), of 16384 558 us with it and
// 439 without (3.8 and 3.7 TB/s).
#include "hm_internal.h"
#include "hm_mx_device.cuh"
#include "hm_ops.h"
#include "hm_ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>

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

}  // namespace

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
