// MXFP8 quantization of activations, gradients and weights along either axis.
//
// y = x * row * col (fp32); per block of 32 (or 128) elements along an axis,
// e = clamp(floor(log2 amax) - 8, -127, 127), codes E4M3_RNE(y 2^-e), scale
// byte e + 127 -- G's rule (hm_mx_device.cuh).  x is read once for both axes:
// the gradient products of a linear layer contract along the tokens, so they
// need the transposed operand of what the forward product uses.
//
// A CTA takes a 128 x 128 tile: the tile's scales are then one 512-byte tile of
// either scale layout.  Memory-bound: bf16 x with both outputs moves
// 2 + 2 (1 + 1/32) bytes per element.
#include "hm_internal.h"
#include "hm_mx_device.cuh"
#include "hm_ops.h"

namespace hm {

namespace {

constexpr int kQThreads = 256;
constexpr int kQTile = 128;

template <bool F32>
__device__ __forceinline__ void load8(const void* x, int64_t at, int left, bool vec, float (&v)[8]) {
    // elements at .. at + 7, those from `left` on being zero
    if (F32) {
        const float* p = static_cast<const float*>(x) + at;
        if (vec && left >= 8) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
            const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k < left ? p[k] : 0.f;
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(x) + at;
        if (vec && left >= 8) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k < left ? __uint_as_float(static_cast<uint32_t>(p[k]) << 16) : 0.f;
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const __grid_constant__ QuantArgs p) {
    extern __shared__ __align__(16) float tile[];  // [128][128], transposed output only
    __shared__ __align__(16) uint8_t s_row[512];
    __shared__ __align__(16) uint8_t s_col[512];
    __shared__ float amax_col[4][kQTile];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ct = blockIdx.x, rt = blockIdx.y;
    const int64_t r0 = rt * kQTile, c0 = ct * kQTile;
    const int64_t cols32 = (p.cols + 31) / 32 * 32, rows32 = (p.rows + 31) / 32 * 32;
    const int c8 = (lane & 15) * 8;
    const int left = static_cast<int>(min(static_cast<int64_t>(8), max(static_cast<int64_t>(0), p.cols - (c0 + c8))));
    float cm[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) cm[k] = p.col_mul && k < left ? p.col_mul[c0 + c8 + k] : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int rl = warp * 16 + i * 2 + (lane >> 4);
        const int64_t r = r0 + rl;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < p.rows && left > 0) {
            load8<F32>(p.x, r * p.ldx + c0 + c8, left, p.vec, v);
            if (p.row_mul) {
                const float rm = p.row_mul[r];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= rm;
            }
            if (p.col_mul) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= cm[k];
            }
        }
        if (p.qt) {
            float4* t4 = reinterpret_cast<float4*>(tile + rl * kQTile + c8);
            t4[0] = make_float4(v[0], v[1], v[2], v[3]);
            t4[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        if (p.q) {
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            if (p.block == 128) {
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
            }
            const int e = mx_scale_exponent(amax);
            const float sc = mx_inv_scale(e);
            const bool live = r < p.rows && c0 + c8 < cols32;
            if (live) {
                const uint32_t lo = cvt_e4m3x2(v[0] * sc, v[1] * sc) | (static_cast<uint32_t>(cvt_e4m3x2(v[2] * sc, v[3] * sc)) << 16);
                const uint32_t hi = cvt_e4m3x2(v[4] * sc, v[5] * sc) | (static_cast<uint32_t>(cvt_e4m3x2(v[6] * sc, v[7] * sc)) << 16);
                *reinterpret_cast<uint2*>(p.q + r * p.ldq + c0 + c8) = make_uint2(lo, hi);
            }
            if ((lane & 3) == 0)
                s_row[(rl & 31) * 16 + (rl >> 5) * 4 + ((lane & 15) >> 2)] = live ? static_cast<uint8_t>(e + 127) : 0;
        }
    }
    __syncthreads();
    if (p.q && threadIdx.x < 32) {
        const int64_t col_tiles = (cols32 + 127) / 128;
        reinterpret_cast<uint4*>(p.s + (rt * col_tiles + ct) * 512)[threadIdx.x] = reinterpret_cast<const uint4*>(s_row)[threadIdx.x];
    }
    if (!p.qt) return;
    // thread: one column, two of its four 32-row blocks
    const int c = threadIdx.x & 127, h = threadIdx.x >> 7;
    const bool col_live = c0 + c < p.cols;
    for (int b = 2 * h; b < 2 * h + 2; ++b) {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) amax = fmaxf(amax, fabsf(tile[(b * 32 + k) * kQTile + c]));
        amax_col[b][c] = amax;
    }
    if (p.block == 128) __syncthreads();
    for (int b = 2 * h; b < 2 * h + 2; ++b) {
        float amax = amax_col[b][c];
        if (p.block == 128)
            amax = fmaxf(fmaxf(amax_col[0][c], amax_col[1][c]), fmaxf(amax_col[2][c], amax_col[3][c]));
        const int e = mx_scale_exponent(amax);
        const float sc = mx_inv_scale(e);
        const bool live = col_live && r0 + b * 32 < rows32;
        s_col[(c & 31) * 16 + (c >> 5) * 4 + b] = live ? static_cast<uint8_t>(e + 127) : 0;
        if (!live) continue;
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float* t = tile + (b * 32 + 4 * k) * kQTile + c;
            w[k] = cvt_e4m3x2(t[0] * sc, t[kQTile] * sc) |
                   (static_cast<uint32_t>(cvt_e4m3x2(t[2 * kQTile] * sc, t[3 * kQTile] * sc)) << 16);
        }
        uint4* out = reinterpret_cast<uint4*>(p.qt + (c0 + c) * p.ldqt + r0 + b * 32);
        out[0] = make_uint4(w[0], w[1], w[2], w[3]);
        out[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int64_t row_tiles = (rows32 + 127) / 128;
        reinterpret_cast<uint4*>(p.st + (ct * row_tiles + rt) * 512)[threadIdx.x] = reinterpret_cast<const uint4*>(s_col)[threadIdx.x];
    }
}

template <bool F32>
cudaError_t launch(const QuantArgs& a, cudaStream_t st) {
    const int smem = a.qt ? kQTile * kQTile * 4 : 0;
    static bool done[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(quantize_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQTile * kQTile * 4);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    const dim3 grid(static_cast<unsigned>((a.cols + 127) / 128), static_cast<unsigned>((a.rows + 127) / 128));
    note_launch();
    quantize_kernel<F32><<<grid, kQThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs& a, int f32, cudaStream_t st) {
    return f32 ? launch<true>(a, st) : launch<false>(a, st);
}

}  // namespace hm
